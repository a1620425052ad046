// Rotary positions and the write into an FP8 cache with a scale for each block
// of tokens and head.
//
//   a = max |x| over the finite values of the new rows of a block and head,
//   need = max(2^-30, the smallest power of two >= a / 448),
//   scale' = need where the rows begin the block, else max(scale, need),
//   code = e4m3(x / scale'); earlier codes of the block: e4m3(code * scale / scale').
//
// A block's scale belongs to all its tokens, so one warp owns a block and head
// for the call: the one at the first of the block's new tokens, which the
// slots alone tell (the block's first slot, or a slot that does not follow the
// token's before it). Warps stand at every window of tokens and every head;
// those whose window begins no block have nothing to do. The owner holds the
// rows of the block in registers while it looks for the largest value, so they
// are read once (longer blocks, of more than 8 KB of rows, are read a second
// time, from the L2). Scales are powers of two: dividing by one is exact, and so
// is moving codes to a larger one, but for those that fall among the subnormals.
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"
#include "gemv_common.cuh"
#include "gemv_rows.cuh"

namespace gemv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQueryTokens = 2;        // tokens whose query rows a thread has in flight (at most 2)

// Cosine and sine of pair `pair` at token `tok`: the angle as a 64-bit fraction of a turn, reduced exactly.
__device__ __forceinline__ float2 turn_of(const RopeParams& p, int64_t tok, int pair) {
    const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
    const int64_t pos = p.positions[axis * p.axis_stride + tok];
    const uint64_t turn = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.freqs[pair]);
    float2 cs;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &cs.y, &cs.x);
    return cs;
}

// The pairs of a group turned: x and y hold their first and second columns, or (interleaved) 2 * VEC neighbouring ones.
template <int VEC, typename Turn>
__device__ __forceinline__ void turn_group(float (&x)[VEC], float (&y)[VEC], bool interleaved, Turn turn) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const float2 cs = turn(j);
        if (!interleaved || VEC == 1) {
            const float u = x[j], v = y[j];
            x[j] = u * cs.x - v * cs.y;
            y[j] = v * cs.x + u * cs.y;
        } else if constexpr (VEC > 1) {
            float& e = j < VEC / 2 ? x[2 * j] : y[2 * j - VEC];
            float& f = j < VEC / 2 ? x[2 * j + 1] : y[2 * j + 1 - VEC];
            const float u = e, v = f;
            e = u * cs.x - v * cs.y;
            f = v * cs.x + u * cs.y;
        }
    }
}

// Four E4M3 codes times `by`, to the nearest codes.
__device__ __forceinline__ uint32_t move_codes(uint32_t v, float by) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(v));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return e4m3x2(a.x * by, a.y * by) | e4m3x2(b.x * by, b.y * by) << 16;
}

// The smallest power of two that is at least top / 448, no smaller than 2^-30; `top`: bits of a finite FP32 >= 0.
__device__ __forceinline__ float scale_for(uint32_t top) {
    // top = m 2^e with 1 <= m < 2; 448 = 1.75 * 2^8. (A subnormal's exponent reads as one below: under the floor.)
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -30) + 127) << 23);
}

// What a warp keeps of a block's rows: groups of 2 * VEC values a lane, 64 values at most.
template <int VEC, bool F32>
constexpr int kHeldGroups = F32 || VEC == 1 ? 8 : 4;

// The blocks that begin among this warp's window of tokens, one head of k or v.
template <int VEC, bool F32>
__device__ __forceinline__ void write_blocks(const RopeParams& p, const BlockScales& b, int window) {
    constexpr int NI = kHeldGroups<VEC, F32>;
    constexpr int es = F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int heads = 2 * p.kv_heads;
    const int64_t wi = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t first = wi / heads * window;
    if (first >= p.tokens) return;
    const int hh = static_cast<int>(wi % heads);
    const bool is_k = hh < p.kv_heads;
    const int of = is_k ? hh : hh - p.kv_heads;
    const int groups = p.head_dim / (2 * VEC), half = p.rot_dim / 2;

    int mine = -1;
    bool begins = false;
    if (lane < window && first + lane < p.tokens) {
        mine = p.slots[first + lane];
        const int before = first + lane > 0 ? p.slots[first + lane - 1] : -1;
        const int in = b.shift >= 0 ? mine & (b.tokens - 1) : mine % b.tokens;
        begins = mine >= 0 && mine < p.num_slots && (in == 0 || before != mine - 1);
    }
    for (uint32_t rest = __ballot_sync(0xffffffffu, begins); rest; rest &= rest - 1) {
        const int at = __ffs(rest) - 1;
        const int64_t tok0 = first + at;
        const int slot = __shfl_sync(0xffffffffu, mine, at);
        const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
        const int place = slot - page * p.page_size;
        const int blk = b.shift >= 0 ? place >> b.shift : place / b.tokens;
        const int held = place - blk * b.tokens;                     // earlier tokens of the block
        // The block's tokens of this call.
        const int most = static_cast<int>(min(static_cast<int64_t>(b.tokens - held), p.tokens - tok0));
        int n = 1;
        while (n < most) {
            const int j = n + lane;
            const uint32_t off = __ballot_sync(0xffffffffu, j >= most || p.slots[tok0 + j] != slot + j);
            n += off ? __ffs(off) - 1 : 32;
            if (off) break;
        }

        float* const scale_at = (is_k ? b.k : b.v) + page * b.page_stride + blk * b.block_stride + of * b.head_stride;
        const float old = held > 0 ? *scale_at : 0.f;
        const int64_t stride = (is_k ? p.k_stride : p.v_stride) * es;
        const char* const src = static_cast<const char*>(is_k ? p.k : p.v) + tok0 * stride + of * p.head_dim * es;
        unsigned char* const block_at = (is_k ? p.kc : p.vc) + page * p.page_stride + of * p.head_stride +
                                        (place - held) * p.slot_stride;
        const int total = n * groups;                                // groups of the block's rows, token by token

        float x[NI][VEC], y[NI][VEC];
        auto place_of = [&](int u, int& tk, int& c0, int& c1, int& gi) {
            tk = u / groups;
            gi = u - tk * groups;
            const bool split = gi * VEC < half && !p.interleaved;
            c0 = split ? gi * VEC : gi * 2 * VEC;
            c1 = split ? half + gi * VEC : gi * 2 * VEC + VEC;
        };
        auto load = [&](int base) {
            Cols<VEC, F32> a[NI], c[NI];
            int tk, c0, c1, gi;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int u = base + i * 32 + lane;
                if (u < total) {
                    place_of(u, tk, c0, c1, gi);
                    a[i].load(src + tk * stride, c0);
                    c[i].load(src + tk * stride, c1);
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int u = base + i * 32 + lane;
                if (u < total) {
                    place_of(u, tk, c0, c1, gi);
                    a[i].values(x[i]);
                    c[i].values(y[i]);
                    if (is_k && gi * VEC < half)
                        turn_group<VEC>(x[i], y[i], p.interleaved, [&](int j) { return turn_of(p, tok0 + tk, gi * VEC + j); });
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[i][j] = y[i][j] = 0.f;
                }
            }
        };
        uint32_t top = 0;
        auto largest = [&](float v) {
            const uint32_t bits = __float_as_uint(v) & 0x7fffffffu;
            top = max(top, bits < 0x7f800000u ? bits : 0u);
        };
        int base = 0;
        while (true) {
            load(base);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    largest(x[i][j]);
                    largest(y[i][j]);
                }
            if (base + NI * 32 >= total) break;
            base += NI * 32;
        }
        const float need = scale_for(__reduce_max_sync(0xffffffffu, top));
        const float scale = held > 0 ? fmaxf(old, need) : need;
        if (held > 0 && scale > old) {                               // earlier tokens move to the new scale
            const float by = old / scale;
            const int per = p.head_dim / 16;
            for (int v = lane; v < held * per; v += 32) {
                const int tk = v / per;
                uint4* const c = reinterpret_cast<uint4*>(block_at + tk * p.slot_stride + (v - tk * per) * 16);
                uint4 w = *c;
                w.x = move_codes(w.x, by);
                w.y = move_codes(w.y, by);
                w.z = move_codes(w.z, by);
                w.w = move_codes(w.w, by);
                *c = w;
            }
        }
        if (lane == 0) *scale_at = scale;
        // The reciprocal, or 0 where the scale is no power of two, or one whose reciprocal FP32 does not hold.
        const uint32_t bits = __float_as_uint(scale), e = bits >> 23 & 255u;
        const float inv = (bits & 0x7fffffu) == 0u && e > 1u && e < 253u ? __frcp_rn(scale) : 0.f;
        while (true) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int u = base + i * 32 + lane;
                if (u < total) {
                    int tk, c0, c1, gi;
                    place_of(u, tk, c0, c1, gi);
                    unsigned char* const to = block_at + (held + tk) * p.slot_stride;
                    store_fp8<VEC>(to, c0, x[i], scale, inv);
                    store_fp8<VEC>(to, c1, y[i], scale, inv);
                }
            }
            if (base == 0) break;
            base -= NI * 32;
            load(base);
        }
    }
}

// Query rows of TT tokens, `visit` heads a CTA: as gemv_rope turns them.
template <int VEC, bool F32, int TT>
__device__ __forceinline__ void turn_queries(const RopeParams& p, int64_t tok0, int part, int visit) {
    constexpr int GAP = VEC > 1 ? 2 : 0;                             // a warp's groups lie in different banks
    __shared__ __align__(16) float2 s_turn[TT][GEMV_MAX_HEAD_DIM / 2 / VEC * (VEC + GAP)];
    constexpr int es = F32 ? 4 : 2;
    const int groups = p.head_dim / (2 * VEC), half = p.rot_dim / 2;
    const int hy = static_cast<int>(threadIdx.x) / groups, gi = threadIdx.x - hy * groups;
    const int h = part * visit + hy;
    const bool is_head = hy < visit && h < p.q_heads;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TT), p.tokens - tok0));
    const bool turned = gi * VEC < half;
    const int c0 = turned && !p.interleaved ? gi * VEC : gi * 2 * VEC;
    const int c1 = turned && !p.interleaved ? half + gi * VEC : gi * 2 * VEC + VEC;
    Cols<VEC, F32> a[TT], c[TT];
    int slot[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        if (is_head && i < tokens) {
            const char* const row = static_cast<const char*>(p.q) + ((tok0 + i) * p.q_stride + h * p.head_dim) * es;
            a[i].load(row, c0);
            c[i].load(row, c1);
        }
        slot[i] = i < tokens ? p.slots[tok0 + i] : -1;
    }
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = TT > 1 && i >= half ? 1 : 0, pair = i - t * half;
        s_turn[t][pair + pair / VEC * GAP] = turn_of(p, tok0 + t, pair);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        if (!is_head || slot[i] < 0 || slot[i] >= p.num_slots) continue;   // a padding row: nothing of it is written
        float x[VEC], y[VEC];
        a[i].values(x);
        c[i].values(y);
        const float2* const cs = s_turn[i] + gi * (VEC + GAP);
        if (turned) turn_group<VEC>(x, y, p.interleaved, [&](int j) { return cs[j]; });
        uint16_t* const o = p.q_out + (tok0 + i) * p.q_out_stride + h * p.head_dim;
        store_bf16<VEC>(o, c0, x);
        store_bf16<VEC>(o, c1, y);
    }
}

// CTAs up to kv_ctas write blocks, the others turn queries.
template <int VEC, bool F32, int TT>
__global__ void __launch_bounds__(kThreads) append_blocks_kernel(const __grid_constant__ RopeParams p,
                                                                 const __grid_constant__ BlockScales b, int window,
                                                                 unsigned kv_ctas, int parts, int visit) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    if (blockIdx.x < kv_ctas) {
        write_blocks<VEC, F32>(p, b, window);
    } else {
        const unsigned q = blockIdx.x - kv_ctas, at = q / parts;
        turn_queries<VEC, F32, TT>(p, static_cast<int64_t>(at) * TT, static_cast<int>(q - at * parts), visit);
    }
}

template <int VEC, bool F32, int TT>
cudaError_t launch_one(const RopeParams& p, const BlockScales& b, int window, int parts, int visit, cudaStream_t s,
                       bool pdl) {
    const int64_t warps = (static_cast<int64_t>(p.tokens) + window - 1) / window * 2 * p.kv_heads;
    const int64_t kv = (warps + kWarps - 1) / kWarps, q = (static_cast<int64_t>(p.tokens) + TT - 1) / TT * parts;
    if (kv + q > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kv + q), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, append_blocks_kernel<VEC, F32, TT>, p, b, window, static_cast<unsigned>(kv), parts,
                              visit);
}

template <int VEC, bool F32>
cudaError_t launch_shape(const RopeParams& p, const BlockScales& b, int sm_count, cudaStream_t s, bool pdl) {
    const int groups = p.head_dim / (2 * VEC), most = kThreads / groups;   // query heads of a CTA
    const int parts = (p.q_heads + most - 1) / most, visit = (p.q_heads + parts - 1) / parts;
    const int window = p.tokens > 4 * sm_count ? 4 : 1;
    if (static_cast<int64_t>(p.tokens) / kQueryTokens * parts < 2 * sm_count)
        return launch_one<VEC, F32, 1>(p, b, window, parts, visit, s, pdl);
    return launch_one<VEC, F32, kQueryTokens>(p, b, window, parts, visit, s, pdl);
}

}  // namespace

cudaError_t launch_append_blocks(const RopeParams& p, const BlockScales& b, int sm_count, cudaStream_t s, bool pdl) {
    if (p.rows_f32)
        return p.vec >= 4 ? launch_shape<4, true>(p, b, sm_count, s, pdl) : launch_shape<1, true>(p, b, sm_count, s, pdl);
    return p.vec >= 8 ? launch_shape<8, false>(p, b, sm_count, s, pdl) : launch_shape<1, false>(p, b, sm_count, s, pdl);
}

}  // namespace gemv
