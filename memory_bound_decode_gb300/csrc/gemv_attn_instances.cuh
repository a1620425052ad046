// Launchers of the paged-attention instances: one translation unit per cache
// kind and head size (they compile in parallel), with the same ring sizes.
#pragma once

#include "gemv_attn_kernel.cuh"

namespace gemv {

// Warps and slices in flight per instance: the ring takes about 192 KB of the
// SM's 227 KB, one CTA per SM.
template <int DT, bool FP8>
struct AttnTune {
    static constexpr int kWarps = DT == 256 ? 4 : 8;
    static constexpr int kStages = (DT == 64 ? 6 : 3) * (FP8 && DT > 64 ? 2 : 1);
};

template <int DT, int NB, bool FP8>
int attn_smem() {
    return AttnShape<DT, NB, FP8, AttnTune<DT, FP8>::kWarps, AttnTune<DT, FP8>::kStages>::kSmem;
}

template <int DT, int NB, bool FP8>
cudaError_t attn_prepare_one() {
    return cudaFuncSetAttribute(
        attn_decode_kernel<DT, NB, FP8, AttnTune<DT, FP8>::kWarps, AttnTune<DT, FP8>::kStages>,
        cudaFuncAttributeMaxDynamicSharedMemorySize, attn_smem<DT, NB, FP8>());
}

template <int DT, int NB, bool FP8>
cudaError_t attn_launch_one(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(l.grid), 1, 1);
    cfg.blockDim = dim3(AttnTune<DT, FP8>::kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(attn_smem<DT, NB, FP8>());
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(
        &cfg, attn_decode_kernel<DT, NB, FP8, AttnTune<DT, FP8>::kWarps, AttnTune<DT, FP8>::kStages>, p);
}

// The status word of this translation unit.
inline cudaError_t attn_read_status(unsigned int* bits, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_status, sizeof(unsigned int));
    if (e != cudaSuccess || !reset || *bits == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(unsigned int));
}

// The functions of one translation unit.
#define GEMV_ATTN_UNIT(SUFFIX, DT, FP8, MAXNB)                                                          \
    cudaError_t attn_prepare_##SUFFIX() {                                                               \
        cudaError_t e = attn_prepare_one<DT, 1, FP8>();                                                 \
        if (e == cudaSuccess) e = attn_prepare_one<DT, 2, FP8>();                                       \
        if constexpr (MAXNB == 4)                                                                       \
            if (e == cudaSuccess) e = attn_prepare_one<DT, 4, FP8>();                                   \
        return e;                                                                                       \
    }                                                                                                   \
    cudaError_t attn_launch_##SUFFIX(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) { \
        if (l.nb == 1) return attn_launch_one<DT, 1, FP8>(p, l, s, pdl);                                \
        if constexpr (MAXNB == 4)                                                                       \
            if (l.nb == 4) return attn_launch_one<DT, 4, FP8>(p, l, s, pdl);                            \
        return attn_launch_one<DT, 2, FP8>(p, l, s, pdl);                                               \
    }                                                                                                   \
    cudaError_t attn_status_##SUFFIX(unsigned int* bits, bool reset) { return attn_read_status(bits, reset); }

}  // namespace gemv
