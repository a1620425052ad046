// Tokens of a paged cache back as rows of BF16 or FP32: a value is its code
// times its scale, rounded once.
//
// One pass: codes in, rows out, bound by HBM. A CTA takes kReadRows rows: it
// finds the request of the first among row_start, its threads the pages of one
// row each, then every thread brings one group of eight values (16 bytes of a
// BF16 row) of row after row.
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
constexpr int kReadRows = 16;
constexpr unsigned int kStatusBadPage = 2u;

// Eight E4M3 codes as FP32.
__device__ __forceinline__ void values_of_codes(uint2 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t two = static_cast<uint16_t>((i < 2 ? v.x : v.y) >> (i & 1) * 16);
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 of = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * i] = of.x;
        f[2 * i + 1] = of.y;
    }
}

template <bool FP8, bool F32>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
    __shared__ int64_t s_code[kReadRows], s_scale[kReadRows];        // where a row's codes and scales begin
    __shared__ int s_state[kReadRows];                               // 1: in the pool, 0: zeros, -1: no row
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tid = threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kReadRows;

    // The request of row0: as many as end at it or before it.
    int r = 0;
    for (int i = 0; i < p.requests; i += kReadThreads) {
        const bool past = i + tid < p.requests && p.row_start[i + tid + 1] <= row0;
        const int n = __syncthreads_count(past);
        r += n;
        if (n < kReadThreads) break;
    }
    if (tid < kReadRows) {
        const int64_t row = row0 + tid;
        int state = -1;
        while (r < p.requests && p.row_start[r + 1] <= row) ++r;
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

    const int per_head = p.head_dim / 8, per_pool = p.kv_heads * per_head;
    for (int c = tid; c < 2 * per_pool; c += kReadThreads) {
        const int which = c >= per_pool ? 1 : 0, in = c - which * per_pool, head = in / per_head;
        unsigned char* const out = p.out[which];
        if (!out) continue;
        const unsigned char* const from = p.pool[which] + head * p.head_stride + (in - head * per_head) * (FP8 ? 8 : 16);
        const float* const scales = FP8 && p.scale[which] ? p.scale[which] + head * p.scale_head_stride : nullptr;
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            const int state = s_state[i];
            if (state < 0) continue;
            float f[8] = {};
            if (state > 0) {
                if constexpr (FP8) {
                    values_of_codes(*reinterpret_cast<const uint2*>(from + s_code[i]), f);
                    const float scale = scales ? scales[s_scale[i]] : 1.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= scale;
                } else {
                    unpack8(*reinterpret_cast<const uint4*>(from + s_code[i]), f);
                }
            }
            unsigned char* const to = out + (row0 + i) * p.out_stride[which];
            if constexpr (F32) {
                float4* const o = reinterpret_cast<float4*>(to) + in * 2;
                o[0] = make_float4(f[0], f[1], f[2], f[3]);
                o[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
                store_bf16<8>(to, in * 8, f);
            }
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
