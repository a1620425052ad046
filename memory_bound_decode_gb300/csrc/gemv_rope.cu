// Rotary positions of q and k, and the write of k and v into the paged cache.
//
//   angle(t, i) = position(axis(i), t) * inv_freq(i)
//   (a, b) -> (a cos - b sin, b cos + a sin)      for the two columns of pair i
//
// One pass over the rows: each is read once, turned in FP32 and rounded once
// to the type it is stored in. Bound by HBM for prompts and by the launch for
// single tokens.
//
// A thread keeps one group of four pairs for all the heads it visits, so the
// sine and cosine of a pair are computed once per thread and visit, while the
// loads of its heads are in flight. The angle is reduced exactly: freqs holds
// inv_freq / (2 pi) as a 64-bit fraction of a turn, so position * freqs modulo
// 2^64 is the angle's fraction of a turn however far the position is, and
// sinpi / cospi of it need no further reduction (FP32 alone would be off by
// 0.03 radians at position 2^20).
#include <cstdint>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gemv_attn_internal.h"

namespace gemv {
namespace {

constexpr int kRopeThreads = 256;

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

// N values from column c of a row in FP32 or BF16.
template <int N, bool F32>
__device__ __forceinline__ void load_cols(float (&f)[N], const void* row, int c) {
    if constexpr (F32) {
        const float* s = static_cast<const float*>(row) + c;
        if constexpr (N == 4) {
            const float4 v = *reinterpret_cast<const float4*>(s);
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else {
            f[0] = *s;
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(row) + c;
        if constexpr (N == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(s);
            f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
            f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
        } else {
            f[0] = __uint_as_float(static_cast<uint32_t>(*s) << 16);
        }
    }
}

template <int N>
__device__ __forceinline__ void store_bf16(void* row, int c, const float (&f)[N]) {
    uint16_t* d = static_cast<uint16_t*>(row) + c;
    if constexpr (N == 4) *reinterpret_cast<uint2*>(d) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    else *d = static_cast<uint16_t>(pack2(f[0], 0.f));
}

// Codes of value / scale. The quotient is rounded to FP32 before it is rounded
// to E4M3: the plain order of operations, and with a scale that is a power of
// two (the usual choice) the quotient is exact.
template <int N>
__device__ __forceinline__ void store_fp8(void* row, int c, const float (&f)[N], float scale) {
    unsigned char* d = static_cast<unsigned char*>(row) + c;
    if constexpr (N == 4)
        *reinterpret_cast<uint32_t*>(d) = e4m3x2(__fdiv_rn(f[0], scale), __fdiv_rn(f[1], scale)) |
                                          e4m3x2(__fdiv_rn(f[2], scale), __fdiv_rn(f[3], scale)) << 16;
    else
        *d = static_cast<unsigned char>(e4m3x2(__fdiv_rn(f[0], scale), 0.f));
}

// VEC pairs per group (4, or 1 where the layout allows no wider access).
// Block (x, y): token x, heads from y * (heads of a visit) * PASS.
template <int VEC, bool F32, int PASS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int groups = p.head_dim / (2 * VEC);
    const int visit = kRopeThreads / groups;              // heads of one visit
    const int gi = threadIdx.x % groups, hv = threadIdx.x / groups;
    if (hv >= visit) return;
    const int64_t tok = blockIdx.x;
    int64_t slot = tok;
    if (p.slots) {
        slot = p.slots[tok];
        if (slot < 0 || slot >= p.num_slots) return;      // a padding row: nothing of it is written
    }
    const int heads = p.q_heads + p.kv_heads * (p.v ? 2 : 1);
    const int half = p.rot_dim / 2;
    const bool turned = gi * VEC < half;
    // Columns of the group's two halves: the first and second columns of its pairs (half split), or its
    // 2 * VEC neighbouring columns (interleaved pairs, and columns past rot_dim, which are copied).
    const int c0 = turned && !p.interleaved ? gi * VEC : gi * 2 * VEC;
    const int c1 = turned && !p.interleaved ? half + gi * VEC : gi * 2 * VEC + VEC;

    float a[PASS][VEC], b[PASS][VEC];
    const int h0 = blockIdx.y * visit * PASS + hv;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
        const int h = h0 + i * visit;
        if (h >= heads) break;
        constexpr int es = F32 ? 4 : 2;
        const char* row;
        if (h < p.q_heads)
            row = static_cast<const char*>(p.q) + (tok * p.q_stride + static_cast<int64_t>(h) * p.head_dim) * es;
        else if (h < p.q_heads + p.kv_heads)
            row = static_cast<const char*>(p.k) +
                  (tok * p.k_stride + static_cast<int64_t>(h - p.q_heads) * p.head_dim) * es;
        else
            row = static_cast<const char*>(p.v) +
                  (tok * p.v_stride + static_cast<int64_t>(h - p.q_heads - p.kv_heads) * p.head_dim) * es;
        load_cols<VEC, F32>(a[i], row, c0);
        load_cols<VEC, F32>(b[i], row, c1);
    }

    float cs[VEC], sn[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        cs[j] = 1.f;
        sn[j] = 0.f;
        if (turned) {
            const int pair = gi * VEC + j;
            const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
            const int64_t pos = p.positions[axis * p.axis_stride + tok];
            const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.freqs[pair]);
            sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[j], &cs[j]);
        }
    }

#pragma unroll
    for (int i = 0; i < PASS; ++i) {
        const int h = h0 + i * visit;
        if (h >= heads) break;
        const bool is_v = h >= p.q_heads + p.kv_heads;
        if (turned && !is_v) {
            if (!p.interleaved || VEC == 1) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float x = a[i][j], y = b[i][j];
                    a[i][j] = x * cs[j] - y * sn[j];
                    b[i][j] = y * cs[j] + x * sn[j];
                }
            } else if constexpr (VEC == 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {             // pairs 0, 1 in a, pairs 2, 3 in b
                    float& u = j < 2 ? a[i][2 * j] : b[i][2 * j - 4];
                    float& v = j < 2 ? a[i][2 * j + 1] : b[i][2 * j - 3];
                    const float x = u, y = v;
                    u = x * cs[j] - y * sn[j];
                    v = y * cs[j] + x * sn[j];
                }
            }
        }
        if (h < p.q_heads) {
            uint16_t* o = p.q_out + tok * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim;
            store_bf16<VEC>(o, c0, a[i]);
            store_bf16<VEC>(o, c1, b[i]);
        } else {
            const int kh = is_v ? h - p.q_heads - p.kv_heads : h - p.q_heads;
            const int64_t page = slot / p.page_size;
            unsigned char* o = (is_v ? p.vc : p.kc) + page * p.page_stride + kh * p.head_stride +
                               (slot - page * p.page_size) * p.slot_stride;
            if (p.fp8) {
                const float* sc = is_v ? p.v_scale : p.k_scale;
                const float scale = sc ? sc[kh] : 1.f;
                store_fp8<VEC>(o, c0, a[i], scale);
                store_fp8<VEC>(o, c1, b[i], scale);
            } else {
                store_bf16<VEC>(o, c0, a[i]);
                store_bf16<VEC>(o, c1, b[i]);
            }
        }
    }
}

template <int VEC, bool F32, int PASS>
cudaError_t launch_one(const RopeParams& p, cudaStream_t s, bool pdl) {
    const int visit = kRopeThreads / (p.head_dim / (2 * VEC)) * PASS;
    const int heads = p.q_heads + p.kv_heads * (p.v ? 2 : 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.tokens), static_cast<unsigned>((heads + visit - 1) / visit), 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rope_kernel<VEC, F32, PASS>, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t s, bool pdl) {
    if (!p.vec)
        return p.rows_f32 ? launch_one<1, true, 1>(p, s, pdl) : launch_one<1, false, 1>(p, s, pdl);
    const int visit = kRopeThreads / (p.head_dim / 8);
    const int heads = p.q_heads + p.kv_heads * (p.v ? 2 : 1);
    const int64_t blocks = static_cast<int64_t>(p.tokens) * ((heads + visit - 1) / visit);
    // Few tokens: one head per thread, so that more SMs share the latency.
    if (blocks <= 8 * static_cast<int64_t>(sm_count))
        return p.rows_f32 ? launch_one<4, true, 1>(p, s, pdl) : launch_one<4, false, 1>(p, s, pdl);
    return p.rows_f32 ? launch_one<4, true, 3>(p, s, pdl) : launch_one<4, false, 3>(p, s, pdl);
}

}  // namespace gemv
