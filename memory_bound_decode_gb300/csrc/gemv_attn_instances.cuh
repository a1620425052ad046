// Launchers of the paged-attention instances: one translation unit per cache
// kind and head size (they compile in parallel), with the same ring sizes.
#pragma once

#include "gemv_attn_kernel.cuh"

namespace gemv {

template <int DT, int NB, bool FP8, bool BLOCK, bool TMA>
cudaError_t attn_prepare_form() {
    return cudaFuncSetAttribute(attn_decode_kernel<DT, NB, FP8, TMA, BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnShape<DT, NB, FP8, TMA, BLOCK>::kSmem);
}

template <int DT, int NB, bool FP8, bool BLOCK>
cudaError_t attn_prepare_one() {
    const cudaError_t e = attn_prepare_form<DT, NB, FP8, BLOCK, true>();
    return e == cudaSuccess ? attn_prepare_form<DT, NB, FP8, BLOCK, false>() : e;
}

template <int DT, int NB, bool FP8, bool BLOCK, bool TMA>
cudaError_t attn_launch_form(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) {
    using S = AttnShape<DT, NB, FP8, TMA, BLOCK>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(l.grid), 1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(S::kSmem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<DT, NB, FP8, TMA, BLOCK>, p);
}

template <int DT, int NB, bool FP8, bool BLOCK>
cudaError_t attn_launch_one(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) {
    return p.tma ? attn_launch_form<DT, NB, FP8, BLOCK, true>(p, l, s, pdl)
                 : attn_launch_form<DT, NB, FP8, BLOCK, false>(p, l, s, pdl);
}

// The status word of this translation unit.
inline cudaError_t attn_read_status(unsigned int* bits, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(unsigned int));
    if (e != cudaSuccess || !reset || *bits == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(unsigned int));
}

// The functions of one translation unit.
#define GEMV_ATTN_UNIT(SUFFIX, DT, FP8, BLOCK, MAXNB)                                                   \
    cudaError_t attn_prepare_##SUFFIX() {                                                               \
        cudaError_t e = attn_prepare_one<DT, 1, FP8, BLOCK>();                                          \
        if (e == cudaSuccess) e = attn_prepare_one<DT, 2, FP8, BLOCK>();                                \
        if constexpr (MAXNB == 4)                                                                       \
            if (e == cudaSuccess) e = attn_prepare_one<DT, 4, FP8, BLOCK>();                            \
        return e;                                                                                       \
    }                                                                                                   \
    cudaError_t attn_launch_##SUFFIX(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) { \
        if (l.nb == 1) return attn_launch_one<DT, 1, FP8, BLOCK>(p, l, s, pdl);                         \
        if constexpr (MAXNB == 4)                                                                       \
            if (l.nb == 4) return attn_launch_one<DT, 4, FP8, BLOCK>(p, l, s, pdl);                     \
        return attn_launch_one<DT, 2, FP8, BLOCK>(p, l, s, pdl);                                        \
    }                                                                                                   \
    cudaError_t attn_status_##SUFFIX(unsigned int* bits, bool reset) { return attn_read_status(bits, reset); }

}  // namespace gemv
