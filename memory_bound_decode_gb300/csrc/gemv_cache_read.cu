// Tokens of a paged cache back as rows of BF16 or FP32: a value is the FP32
// product of its code and its scale (exact where that is a power of two),
// rounded to BF16 where the rows are.
//
// One pass: codes in, rows out, bound by HBM: 16 requests of up to 4,096 tokens
// (8 heads of 128 to BF16 rows, 201 MB) 32.3 us, 6.2 TB/s; FP32 rows of 840 MB
// in all 129 us, 6.5 TB/s; 300 tokens 3.2 us in a replayed graph, of which 2 are the launch.
// A CTA takes kReadRows rows (4, 8, 16, 32: 35.6, 34.0, 34.8, 35.8 us): it
// finds the request of the first among row_start, its threads the pages of one
// row each, then every thread brings the same 16 bytes of row after row.
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"
#include "gemv_common.cuh"
#include "gemv_rows.cuh"

namespace gemv {

static __device__ unsigned int g_read_status;

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadRows = 8;
constexpr unsigned int kStatusBadPage = 2u;

// N values of a cache as they come: codes, or BF16.
template <int N, bool FP8>
struct Held {
    static constexpr int kBytes = N * (FP8 ? 1 : 2);
    uint32_t w[kBytes / 4];
    __device__ __forceinline__ void load(const unsigned char* at) {
        if constexpr (kBytes == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(at));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(at));
            w[0] = v.x; w[1] = v.y;
        } else {
            w[0] = __ldcs(reinterpret_cast<const unsigned int*>(at));
        }
    }
    __device__ __forceinline__ void values(float scale, float (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (FP8) {
                uint32_t h;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[i / 2] >> (i & 1) * 16)));
                const float2 of = __half22float2(*reinterpret_cast<const __half2*>(&h));
                f[2 * i] = of.x * scale;
                f[2 * i + 1] = of.y * scale;
            } else {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
};

template <bool FP8, bool F32>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
    __shared__ int64_t s_code[kReadRows], s_scale[kReadRows];        // where a row's codes and scales begin
    __shared__ int s_state[kReadRows];                               // 1: in the pool, 0: zeros, -1: no row
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;

    // The request of row0: as many as end at it or before it, searched kReadThreads at a time (one after the other: 4,096
    // requests of 16 tokens 69.4 us, so 62.3, 65,536 of two 716 and 130).
    int r = 0, step = 1;
    while (static_cast<int64_t>(step) * kReadThreads < p.requests) step *= kReadThreads;
    for (; step > 0; step /= kReadThreads) {
        const int64_t i = r + static_cast<int64_t>(tid + 1) * step;
        r += step * __syncthreads_count(i <= p.requests && p.row_start[i] <= row0);
    }
    if (tid < kReadRows) {
        const int64_t row = row0 + tid;
        int state = -1;
        // The row's own, a request or more on: steps that double, then halve.
        auto past = [&](int64_t i) { return i <= p.requests && p.row_start[i] <= row; };
        int64_t hop = 1;
        for (; past(r + hop); hop *= 2) r += static_cast<int>(hop);
        while ((hop /= 2) > 0)
            if (past(r + hop)) r += static_cast<int>(hop);
        if (row < p.rows && r < p.requests) {
            const int64_t tok = (p.begin ? p.begin[r] : 0) + row - p.row_start[r];
            state = 0;
            if (tok >= 0 && tok < static_cast<int64_t>(p.table_width) * p.page_size) {
                const int t = static_cast<int>(tok);
                const int at = p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size, place = t - at * p.page_size;
                const int page = p.table[r * p.table_stride + at];
                if (page >= 0 && page < p.num_pages) {
                    const int blk = p.block_shift >= 0 ? place >> p.block_shift : place / p.block_tokens;
                    s_code[tid] = page * p.page_stride + place * p.slot_stride;
                    s_scale[tid] = page * p.scale_page_stride + blk * p.scale_block_stride;
                    state = 1;
                }
            }
            if (state == 0) atomicOr(&g_read_status, kStatusBadPage);
        }
        s_state[tid] = state;
    }
    __syncthreads();

    // A thread's 16 bytes of a row (eight BF16 values, four FP32 ones), all of the CTA's rows in flight. What is written
    // leaves the L2 first (16 x 4,096 tokens 33.7 -> 32.3 us).
    constexpr int N = F32 ? 4 : 8;
    const int per_head = p.head_dim / N, per_pool = p.kv_heads * per_head;
    for (int c = tid; c < 2 * per_pool; c += kReadThreads) {
        const int which = c >= per_pool ? 1 : 0, in = c - which * per_pool, head = in / per_head;
        if (!p.out[which]) continue;
        unsigned char* const out = p.out[which] + row0 * p.out_stride[which] + in * 16;
        const unsigned char* const from = p.pool[which] + head * p.head_stride + (in - head * per_head) * Held<N, FP8>::kBytes;
        const float* const scales = FP8 && p.scale[which] ? p.scale[which] + head * p.scale_head_stride : nullptr;
        Held<N, FP8> v[kReadRows];
        float scale[kReadRows];
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            scale[i] = 1.f;
            if (s_state[i] > 0) {
                v[i].load(from + s_code[i]);
                if (scales) scale[i] = scales[s_scale[i]];
            }
        }
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            const int state = s_state[i];
            if (state < 0) continue;
            float f[N];
            v[i].values(scale[i], f);
            if (state == 0) {
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = 0.f;
            }
            unsigned char* const to = out + i * p.out_stride[which];
            if constexpr (F32)
                __stcs(reinterpret_cast<float4*>(to), make_float4(f[0], f[1], f[2], f[3]));
            else
                __stcs(reinterpret_cast<uint4*>(to),
                       make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
        }
    }
}

template <bool FP8, bool F32>
cudaError_t launch_one(const ReadParams& p, cudaStream_t s, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.rows + kReadRows - 1) / kReadRows), 1, 1);
    cfg.blockDim = dim3(kReadThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, cache_read_kernel<FP8, F32>, p);
}

}  // namespace

cudaError_t prepare_read() {
    cudaFuncAttributes a;                                            // (asking for them loads the kernel)
    cudaError_t e = cudaFuncGetAttributes(&a, cache_read_kernel<true, true>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, cache_read_kernel<true, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, cache_read_kernel<false, true>);
    return e == cudaSuccess ? cudaFuncGetAttributes(&a, cache_read_kernel<false, false>) : e;
}

cudaError_t launch_read(const ReadParams& p, cudaStream_t s, bool pdl) {
    if (p.fp8) return p.rows_f32 ? launch_one<true, true>(p, s, pdl) : launch_one<true, false>(p, s, pdl);
    return p.rows_f32 ? launch_one<false, true>(p, s, pdl) : launch_one<false, false>(p, s, pdl);
}

cudaError_t read_read_status(unsigned int* bits, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_read_status, sizeof(unsigned int));
    if (e != cudaSuccess || !reset || *bits == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_read_status, &zero, sizeof(unsigned int));
}

}  // namespace gemv
