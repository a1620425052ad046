// Rotary positions of q and k, and the write of k and v into the paged cache.
//
//   angle(t, i) = position(axis(i), t) * inv_freq(i)
//   (a, b) -> (a cos - b sin, b cos + a sin)      for the two columns of pair i
//
// One pass over the rows: each is read once, turned in FP32 and rounded once
// to the type it is stored in. Bound by HBM for prompts and by the launch for
// single tokens.
//
// A thread takes one group of eight (FP32: four) pairs, 32 bytes of a row, of
// one head for kRopeTokens tokens, whose loads all go out first; while they
// are in flight the block computes the sine and cosine of its tokens' pairs,
// once each. A block lives for a chain of latencies (positions, sines, a
// barrier, stores), so what bounds it is the bytes it has in flight meanwhile
// against the blocks an SM holds. Measured (before the sines were laid out
// without bank conflicts) with 1, 2, 4 and 8 tokens: 8,100 image patches of
// 2 x 16 heads of 80 columns 22.1, 17.2, 18.0, 22.0 us, a prompt of 4,096
// tokens of 48 FP32 heads 27.1, 23.0, 25.4, 30.8 us. Now 14.7 us (5.6 TB/s)
// and 22.8 (6.6 TB/s).
//
// The angle is reduced exactly: freqs holds inv_freq / (2 pi) as a 64-bit
// fraction of a turn, so position * freqs modulo 2^64 is the angle's fraction
// of a turn however far the position is, and sinpi / cospi of it need no
// further reduction (FP32 alone would be off by 0.03 radians at position 2^20).
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"
#include "gemv_common.cuh"

namespace gemv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 2;         // tokens whose rows a thread has in flight (at most 2)

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two values to E4M3 codes, to nearest, values past 448 to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// N values from column c of a row in FP32 or BF16, as they come.
template <int N, bool F32>
struct Cols {
    static constexpr int kWords = N == 1 ? 1 : 4;         // N values of a wide load take 16 bytes
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char* row, int c) {
        if constexpr (N > 1) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + c * (F32 ? 4 : 2));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (F32) {
            w[0] = reinterpret_cast<const uint32_t*>(row)[c];
        } else {
            w[0] = reinterpret_cast<const uint16_t*>(row)[c];
        }
    }
    __device__ __forceinline__ void values(float (&f)[N]) const {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (N > 1) {
            unpack8(make_uint4(w[0], w[1], w[2], w[3]), f);
        } else {
            f[0] = bf16_lo(w[0]);
        }
    }
};

template <int N>
__device__ __forceinline__ void store_bf16(void* row, int c, const float (&f)[N]) {
    uint16_t* d = static_cast<uint16_t*>(row) + c;
    if constexpr (N == 8)
        *reinterpret_cast<uint4*>(d) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    else if constexpr (N == 4)
        *reinterpret_cast<uint2*>(d) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    else
        *d = static_cast<uint16_t>(pack2(f[0], 0.f));
}

// Codes of value / scale, the quotient in FP32: times the reciprocal where that is exact (a scale that is a power of
// two, the usual choice), else (inv = 0) by division.
template <int N>
__device__ __forceinline__ void store_fp8(void* row, int c, const float (&f)[N], float scale, float inv) {
    unsigned char* d = static_cast<unsigned char*>(row) + c;
    float x[N];
    if (inv != 0.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = f[i] * inv;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __fdiv_rn(f[i], scale);
    }
    if constexpr (N == 8)
        *reinterpret_cast<uint2*>(d) = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16,
                                                  e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    else if constexpr (N == 4)
        *reinterpret_cast<uint32_t*>(d) = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    else
        *d = static_cast<unsigned char>(e4m3x2(x[0], 0.f));
}

// VEC pairs per group (8 of BF16 rows, 4 of FP32 ones, or 1 where the layout allows no wider access).
// Block (x, y): tokens x * TT .., heads y * blockDim.y ..; thread (i, j): group i of the block's head j.
template <int VEC, bool F32, bool FP8, int TT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    // Cosine and sine of the tokens' pairs, those of a thread 16 bytes apart from the next one's: the groups that a
    // warp reads lie in different banks (image patches 16.9 -> 14.6 us, the FP8 append 8.1 -> 7.2).
    constexpr int GAP = VEC > 1 ? 2 : 0;
    __shared__ __align__(16) float2 s_turn[TT][GEMV_MAX_HEAD_DIM / 2 / VEC * (VEC + GAP)];
    pdl_launch_dependents();
    const int gi = threadIdx.x, h = blockIdx.y * blockDim.y + threadIdx.y;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TT;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TT), p.tokens - tok0));
    const int half = p.rot_dim / 2;
    const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
    const bool is_head = h < p.q_heads + p.kv_heads * (p.v ? 2 : 1);
    const int of = is_q ? h : is_k ? h - p.q_heads : h - p.q_heads - p.kv_heads;
    // Columns of the group's two halves: the first and second columns of its pairs (half split), or its
    // 2 * VEC neighbouring columns (interleaved pairs, and columns past rot_dim, which are copied).
    const bool turned = gi * VEC < half;
    const int c0 = turned && !p.interleaved ? gi * VEC : gi * 2 * VEC;
    const int c1 = turned && !p.interleaved ? half + gi * VEC : gi * 2 * VEC + VEC;
    pdl_wait_prerequisites();

    Cols<VEC, F32> a[TT], b[TT];
    {
        constexpr int es = F32 ? 4 : 2;
        const int64_t stride = (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) * es;
        const char* row = static_cast<const char*>(is_q ? p.q : is_k ? p.k : p.v) + tok0 * stride + of * p.head_dim * es;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (is_head && i < tokens) {
                a[i].load(row, c0);
                b[i].load(row, c1);
            }
            row += stride;
        }
    }
    const int lane = threadIdx.y * blockDim.x + gi;
    for (int i = lane; i < tokens * half; i += blockDim.x * blockDim.y) {
        const int t = TT > 1 && i >= half ? 1 : 0, pair = i - t * half;
        const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
        const int64_t pos = p.positions[axis * p.axis_stride + tok0 + t];
        const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.freqs[pair]);
        float2 cs;
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &cs.y, &cs.x);
        s_turn[t][pair + pair / VEC * GAP] = cs;
    }
    int slot[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) slot[i] = p.slots && i < tokens ? p.slots[tok0 + i] : 0;
    float scale = 1.f, inv = 1.f;
    if (FP8 && is_head && !is_q) {
        const float* sc = is_k ? p.k_scale : p.v_scale;
        if (sc) scale = sc[of];
        // The reciprocal, or 0 where the scale is no power of two, or one whose reciprocal FP32 does not hold.
        const uint32_t bits = __float_as_uint(scale), e = bits >> 23 & 255u;
        inv = (bits & 0x7fffffu) == 0u && e > 1u && e < 253u ? __frcp_rn(scale) : 0.f;
    }
    __syncthreads();
    if (!is_head) return;

#pragma unroll
    for (int i = 0; i < TT; ++i) {
        if (i >= tokens) break;
        int64_t place = (tok0 + i) * p.page_stride;       // of the token in the cache
        if (p.slots) {
            if (slot[i] < 0 || slot[i] >= p.num_slots) continue;   // a padding row: nothing of it is written
            const int page = p.page_shift >= 0 ? slot[i] >> p.page_shift : slot[i] / p.page_size;
            place = page * p.page_stride + (slot[i] - page * p.page_size) * p.slot_stride;
        }
        float x[VEC], y[VEC];
        a[i].values(x);
        b[i].values(y);
        if (turned && (is_q || is_k)) {
            const float2* const cs = s_turn[i] + gi * (VEC + GAP);
            if (!p.interleaved || VEC == 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float u = x[j], v = y[j];
                    x[j] = u * cs[j].x - v * cs[j].y;
                    y[j] = v * cs[j].x + u * cs[j].y;
                }
            } else if constexpr (VEC > 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {           // the first half of the pairs in x, the others in y
                    float& e = j < VEC / 2 ? x[2 * j] : y[2 * j - VEC];
                    float& f = j < VEC / 2 ? x[2 * j + 1] : y[2 * j + 1 - VEC];
                    const float u = e, v = f;
                    e = u * cs[j].x - v * cs[j].y;
                    f = v * cs[j].x + u * cs[j].y;
                }
            }
        }
        if (is_q) {
            uint16_t* o = p.q_out + (tok0 + i) * p.q_out_stride + of * p.head_dim;
            store_bf16<VEC>(o, c0, x);
            store_bf16<VEC>(o, c1, y);
            continue;
        }
        unsigned char* o = (is_k ? p.kc : p.vc) + place + of * p.head_stride;
        if constexpr (FP8) {
            store_fp8<VEC>(o, c0, x, scale, inv);
            store_fp8<VEC>(o, c1, y, scale, inv);
        } else {
            store_bf16<VEC>(o, c0, x);
            store_bf16<VEC>(o, c1, y);
        }
    }
}

template <int VEC, bool F32, bool FP8, int TT>
cudaError_t launch_one(const RopeParams& p, int visit, int blocks, cudaStream_t s, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.tokens) + TT - 1) / TT),
                       static_cast<unsigned>(blocks), 1);
    cfg.blockDim = dim3(static_cast<unsigned>(p.head_dim / (2 * VEC)), static_cast<unsigned>(visit), 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rope_kernel<VEC, F32, FP8, TT>, p);
}

// As few blocks for a token's heads as kRopeThreads allow, equally full; a
// token a block where there are too few tokens to give every SM two blocks of
// kRopeTokens (16 tokens of a decode step: 2.2 us either way, the launch).
template <int VEC, bool F32, bool FP8>
cudaError_t launch_shape(const RopeParams& p, int sm_count, cudaStream_t s, bool pdl) {
    const int heads = p.q_heads + p.kv_heads * (p.v ? 2 : 1), groups = p.head_dim / (2 * VEC);
    const int most = kRopeThreads / groups;               // heads of a block
    const int blocks = (heads + most - 1) / most;
    const int visit = (heads + blocks - 1) / blocks;
    const int64_t full = static_cast<int64_t>(p.tokens) / kRopeTokens * blocks;
    if (full < 2 * sm_count) return launch_one<VEC, F32, FP8, 1>(p, visit, blocks, s, pdl);
    return launch_one<VEC, F32, FP8, kRopeTokens>(p, visit, blocks, s, pdl);
}

template <int VEC, bool F32>
cudaError_t launch_kind(const RopeParams& p, int sm_count, cudaStream_t s, bool pdl) {
    return p.fp8 ? launch_shape<VEC, F32, true>(p, sm_count, s, pdl)
                 : launch_shape<VEC, F32, false>(p, sm_count, s, pdl);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t s, bool pdl) {
    if (p.rows_f32)
        return p.vec >= 4 ? launch_kind<4, true>(p, sm_count, s, pdl) : launch_kind<1, true>(p, sm_count, s, pdl);
    return p.vec >= 8 ? launch_kind<8, false>(p, sm_count, s, pdl) : launch_kind<1, false>(p, sm_count, s, pdl);
}

}  // namespace gemv
