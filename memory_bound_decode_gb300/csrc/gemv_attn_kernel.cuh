// Attention of one new token per request over a paged key-value cache.
//
//   s_j = cap(scale * q . k_j),  p_j = exp(s_j - m),  out = sum_j p_j v_j / sum_j p_j
//
// over the visible tokens j of a request, with the running maximum m and sum
// of a softmax kept in FP32, so K and V are read once and no score is stored.
//
// Work split. A row is one (request, key-value head) pair; its tokens are cut
// into slices of 16. All slices of all rows form one list (request-major), and
// each CTA takes an equal, contiguous range of it, whatever the lengths are:
// the lengths live on the device, so every CTA sums them itself. Inside a CTA
// the warps take the range's slices in turn. A row inside one range is
// finished there; a row cut between CTAs leaves FP32 partial results (output,
// maximum, sum) in the workspace and the CTA that arrives last joins them in
// list order, so the result does not depend on which one that is.
//
// Tiles. The group of query heads that share a key-value head are the narrow
// side (N = 8) of the MMAs, the 16 tokens of a slice (scores) or 16 columns of
// the head (output) the wide one: S^T = K Q^T and O^T = V^T P^T. K and V then
// come straight from shared memory as the A operand (ldmatrix, transposed for
// V), each fetched once, and the running maximum and sum of a head sit in the
// same lanes as its output columns. S^T becomes the B operand of the second
// product by an 8x8 transposition in registers (movmatrix).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gemv_attn_internal.h"

namespace gemv {

static __device__ unsigned int g_attn_status;
constexpr unsigned int kStatusBadPage = 2u;

namespace attn {

__device__ __forceinline__ uint32_t sm_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E4M3 codes (low 16 bits of v) to two FP16 values, exactly.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace attn

// Tokens of request r that its query can reach: its length, cut to what its
// row of the table holds (with a status bit); 0 for an empty request, negative
// for one that has no query row in this call.
__device__ __forceinline__ int attn_len(const AttnParams& p, int r) {
    int len = p.lens[r];
    if (p.token_start) {
        const int a = p.token_start[r], b = p.token_start[r + 1];
        if (b <= a) return -1;
        if (a < 0 || b > p.rows) {
            atomicOr(&g_attn_status, kStatusBadPage);
            return -1;
        }
    }
    if (len > p.max_len) {
        atomicOr(&g_attn_status, kStatusBadPage);
        len = p.max_len;
    }
    return len;
}
__device__ __forceinline__ int64_t attn_row(const AttnParams& p, int r) {
    return p.token_start ? static_cast<int64_t>(p.token_start[r + 1]) - 1 : r;
}
__device__ __forceinline__ int attn_begin(const AttnParams& p, int len) {
    return p.window > 0 && len > p.window ? len - p.window : 0;
}
__device__ __forceinline__ int attn_slices(const AttnParams& p, int len) {
    return len <= 0 ? 0 : (len + kAttnSlice - 1) / kAttnSlice - attn_begin(p, len) / kAttnSlice;
}

// DT: head size of the instance (head_dim <= DT; columns past head_dim are
// zero). NB: blocks of 8 query heads. W: warps. ST: slices in flight per warp.
template <int DT, int NB, bool FP8, int W, int ST>
struct AttnShape {
    static constexpr int kThreads = W * 32;
    static constexpr int kRowBytes = DT * (FP8 ? 1 : 2);
    static constexpr int kSliceBytes = 2 * kAttnSlice * kRowBytes;   // K and V
    static constexpr int kRing = W * ST * kSliceBytes;
    static constexpr int kPartStride = DT + 4;                       // + maximum, sum and two words of padding
    static constexpr int kPart = W * 8 * kPartStride * 4;
    static constexpr int kSmem = kRing + kPart;
};

template <int DT, int NB, bool FP8, int W, int ST>
__global__ void __launch_bounds__(W * 32, 1) attn_decode_kernel(const __grid_constant__ AttnParams p) {
    using S = AttnShape<DT, NB, FP8, W, ST>;
    using namespace attn;
    constexpr int T = S::kThreads;
    constexpr int RB = S::kRowBytes;
    constexpr int CPR = RB / 16;          // 16-byte chunks of a row
    constexpr int KS = DT / 16;           // MMA steps along the head
    constexpr float kNegInf = -INFINITY;
    constexpr float kLog2e = 1.4426950408889634f;

    extern __shared__ __align__(128) unsigned char smem[];
    float* const part_s = reinterpret_cast<float*>(smem + S::kRing);
    __shared__ int32_t s_len[T];
    __shared__ int64_t s_scan[W + 1];
    __shared__ int64_t s_off;
    __shared__ int32_t s_r0;
    __shared__ int32_t s_last;

    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int qt = blockIdx.x % p.qtiles;
    const int cta = blockIdx.x / p.qtiles;
    const int ctas = gridDim.x / p.qtiles;
    const int head0 = qt * NB * 8;                                  // first query head of the group
    const int nh = min(NB * 8, p.group - head0);                    // query heads of this tile

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Requests without a visible token: zeros (nothing to average).
    for (int r = blockIdx.x; r < p.requests; r += gridDim.x) {
        if (p.lens[r] != 0 || attn_len(p, r) != 0) continue;
        const int64_t row = attn_row(p, r);
        const int n4 = p.q_heads * p.head_dim / 4;
        uint2* o = reinterpret_cast<uint2*>(p.out + row * p.out_stride);
        for (int i = tid; i < n4; i += T) o[i] = make_uint2(0, 0);
        if (p.lse)
            for (int i = tid; i < p.q_heads; i += T) p.lse[row * p.q_heads + i] = kNegInf;
    }

    // This CTA's range of the list of slices.
    int64_t mine = 0;
    for (int r = tid; r < p.requests; r += T) mine += attn_slices(p, attn_len(p, r));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_scan[w] = mine;
    if (tid == 0) s_r0 = -1;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) total += s_scan[i];
    total *= p.kv_heads;
    const int64_t quota = max((total + ctas - 1) / ctas, static_cast<int64_t>(W));
    const int64_t f0 = cta * quota;
    if (f0 >= total) return;
    const int cnt = static_cast<int>(min(quota, total - f0));

    // Its first row: the request whose slices contain f0.
    int64_t carry = 0;
    for (int base = 0; base < p.requests; base += T) {
        const int r = base + tid;
        const int n = r < p.requests ? attn_slices(p, attn_len(p, r)) : 0;
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();                                            // s_scan of the step before has been read
        if (lane == 31) s_scan[w] = incl;
        __syncthreads();
        int64_t before = carry;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < w) before += s_scan[i];
            carry += s_scan[i];
        }
        const int64_t lo = (before + incl - n) * p.kv_heads, hi = (before + incl) * p.kv_heads;
        if (lo <= f0 && f0 < hi) {
            s_r0 = r;
            s_off = f0 - lo;
        }
        if (f0 < carry * p.kv_heads) break;                         // the same for all threads
    }
    __syncthreads();
    const int r0 = s_r0;
    if (r0 < 0) return;                                             // only if lens changed under the call
    s_len[tid] = r0 + tid < p.requests ? attn_len(p, r0 + tid) : 0;
    __syncthreads();
    auto len_of = [&](int r) { return r - r0 < T ? s_len[r - r0] : attn_len(p, r); };

    const int ns0 = attn_slices(p, s_len[0]);
    const int h_first = static_cast<int>(s_off / ns0);
    const int s_first = static_cast<int>(s_off - static_cast<int64_t>(h_first) * ns0);

    // ---- copies of K and V into this warp's ring ----
    const uint32_t ring = sm_addr(smem) + static_cast<uint32_t>(w) * ST * S::kSliceBytes;
    const int warp_slices = cnt > w ? (cnt - w + W - 1) / W : 0;
    const int chunks = p.head_dim * (FP8 ? 1 : 2) / 16;
    int pr = r0, ph = h_first, ps = s_first, pns = ns0, plen = s_len[0];
    int issued = 0;
    uint32_t valid_of_stage = 0;          // lane i: the visible tokens of the slice in stage i
    int next_page = -1, next_in = 0;      // lane i < 16: page and place of token i of the next slice
    int next_h = 0;
    auto settle = [&](int step) {         // move the cursor on by `step` slices and look up the pages there
        ps += step;
        while (ps >= pns) {
            ps -= pns;
            if (++ph == p.kv_heads) {
                ph = 0;
                do {
                    if (++pr >= p.requests) {                        // only if lens changed under the call
                        plen = 0;
                        pns = 0x7fffffff;
                        break;
                    }
                    plen = len_of(pr);
                    pns = attn_slices(p, plen);
                } while (pns == 0);
            }
        }
        const int begin = attn_begin(p, plen);
        const int tok = (begin / kAttnSlice + ps) * kAttnSlice + (lane & 15);
        const bool in = tok >= begin && tok < plen;
        const int blk = tok / p.page_size;
        next_in = in ? tok - blk * p.page_size : -1;
        next_page = in ? p.table[pr * p.table_stride + blk] : -1;
        next_h = ph;
    };
    auto issue = [&]() {
        if (issued < warp_slices) {
            const int st = issued % ST;
            int64_t off = -1;
            if (next_in >= 0) {
                if (next_page >= 0 && next_page < p.num_pages)
                    off = next_page * p.page_stride + next_h * p.head_stride + next_in * p.slot_stride;
                else
                    atomicOr(&g_attn_status, kStatusBadPage);
            }
            const uint32_t valid = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
            if (lane == st) valid_of_stage = valid;
            const uint32_t kdst = ring + st * S::kSliceBytes;
#pragma unroll
            for (int i = 0; i < kAttnSlice * CPR / 32; ++i) {
                const int idx = i * 32 + lane, row = idx / CPR, ch = idx % CPR;
                const int64_t o = __shfl_sync(0xffffffffu, off, row);
                const int sw = CPR >= 8 ? row & 7 : (row >> 1) & 3;
                const uint32_t dst = kdst + row * RB + ((ch ^ sw) << 4);
                const int n = o >= 0 && ch < chunks ? 16 : 0;       // 0: the chunk is filled with zeros
                const int64_t at = n ? o + ch * 16 : 0;
                copy16(dst, p.kc + at, n);
                copy16(dst + kAttnSlice * RB, p.vc + at, n);
            }
            ++issued;
            if (issued < warp_slices) settle(W);
        }
        copy_commit();
    };
    if (warp_slices > 0) settle(w);
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue();

    // ---- rows of the range, one after the other ----
    int r = r0, h = h_first, s = s_first, done = 0, li = w, consumed = 0;
    while (done < cnt) {
        const int len = len_of(r);
        const int ns = attn_slices(p, len);
        const int seg = min(ns - s, cnt - done);
        if (seg <= 0) break;
        const int64_t row = attn_row(p, r);
        const int64_t head_at = static_cast<int64_t>(h) * p.group + head0;

        // Query fragments (B operand: 16 columns of the head x 8 heads).
        uint32_t qf[KS][NB][2];
        float col_scale[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const bool in = nb * 8 + g < nh;
            const uint16_t* qp = p.q + row * p.q_stride + (head_at + nb * 8 + g) * p.head_dim;
            if constexpr (!FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int d = ks * 16 + b * 8 + 2 * t;
                        qf[ks][nb][b] = in && d < p.head_dim ? *reinterpret_cast<const uint32_t*>(qp + d) : 0u;
                    }
                col_scale[nb][0] = col_scale[nb][1] = p.scale;
            } else {
                // The FP8 cache is widened to FP16 (exact); q is brought to FP16 by a power of two per head
                // that puts its largest value in [1, 2): what that loses is below 2^-24 of that value.
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int d = ks * 16 + 4 * t;
                    const uint2 v = in && d < p.head_dim ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
                    qf[ks][nb][0] = v.x;
                    qf[ks][nb][1] = v.y;
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(low_bf16(v.x)), fabsf(high_bf16(v.x))),
                                           fmaxf(fabsf(low_bf16(v.y)), fabsf(high_bf16(v.y)))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
                e = top > 0.f ? max(-126, min(126, e)) : 0;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        qf[ks][nb][b] = pack_f16(low_bf16(qf[ks][nb][b]) * down, high_bf16(qf[ks][nb][b]) * down);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                const float ksc = p.scale * (p.k_scale ? p.k_scale[h] : 1.f);
                col_scale[nb][0] = __shfl_sync(0xffffffffu, up, 8 * t) * ksc;
                col_scale[nb][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4) * ksc;
            }
        }

        float m[NB][2], l[NB][2], acc[KS][NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = kNegInf;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[ks][nb][j] = 0.f;
        }

        for (; li < done + seg; li += W) {
            copy_wait<ST - 2>();
            __syncwarp();
            issue();                                                 // into the stage read one step ago
            const int st = consumed % ST;
            ++consumed;
            const uint32_t valid = __shfl_sync(0xffffffffu, valid_of_stage, st);
            const uint32_t kb = ring + st * S::kSliceBytes, vb = kb + kAttnSlice * RB;

            // S^T = K Q^T: rows g and g + 8 are tokens, columns 2t and 2t + 1 heads.
            float sc[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
            const int arow = lane & 15;
            const int asw = CPR >= 8 ? arow & 7 : (arow >> 1) & 3;
#pragma unroll
            for (int c = 0; c < CPR; c += 2) {                       // two 16-byte chunks of the 16 rows
                uint32_t a[4];
                ldsm4(a, kb + arow * RB + (((c + (lane >> 4)) ^ asw) << 4));
                if constexpr (!FP8) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        mma<false>(sc[nb], a[0], a[1], a[2], a[3], qf[c / 2][nb][0], qf[c / 2][nb][1]);
                } else {
                    // Bytes 4t .. 4t + 3 of a chunk: columns 2t, 2t + 1 and 2t + 8, 2t + 9 of the step, by a
                    // permutation of the chunk's columns that q's fragments share.
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t a0 = e4m3_pair(a[2 * x]), a2 = e4m3_pair(a[2 * x] >> 16);
                        const uint32_t a1 = e4m3_pair(a[2 * x + 1]), a3 = e4m3_pair(a[2 * x + 1] >> 16);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma<true>(sc[nb], a0, a1, a2, a3, qf[c + x][nb][0], qf[c + x][nb][1]);
                    }
                }
            }

            // Running maximum and sum, in powers of two.
            uint32_t pb[NB][2], pl[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v = sc[nb][j] * col_scale[nb][j & 1];
                    if (p.softcap > 0.f) v = p.softcap * tanhf(v / p.softcap);
                    v *= kLog2e;
                    x[j] = valid >> (g + (j & 2) * 4) & 1u ? v : kNegInf;
                }
                float corr[2], base[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(x[j], x[j + 2]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[nb][j]);
                    base[j] = top == kNegInf ? 0.f : top;
                    corr[j] = exp2f(m[nb][j] - base[j]);
                    m[nb][j] = top;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = exp2f(x[j] - base[j & 1]);
                l[nb][0] = l[nb][0] * corr[0] + (x[0] + x[2]);
                l[nb][1] = l[nb][1] * corr[1] + (x[1] + x[3]);
                if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        acc[ks][nb][0] *= corr[0];
                        acc[ks][nb][1] *= corr[1];
                        acc[ks][nb][2] *= corr[0];
                        acc[ks][nb][3] *= corr[1];
                    }
                }
                // P as the B operand. FP16 beside an FP8 cache (2^-12 relative). Beside a BF16 cache P has to be
                // BF16, whose 2^-9 would double the rounding error of a BF16 output: it goes in two parts
                // (the rest in a second BF16), 2^-18 together.
                if constexpr (FP8) {
                    pb[nb][0] = transpose8x8(pack_f16(x[0], x[1]));
                    pb[nb][1] = transpose8x8(pack_f16(x[2], x[3]));
                } else {
                    const uint32_t a = pack_bf16(x[0], x[1]), b = pack_bf16(x[2], x[3]);
                    pb[nb][0] = transpose8x8(a);
                    pb[nb][1] = transpose8x8(b);
                    pl[nb][0] = transpose8x8(pack_bf16(x[0] - low_bf16(a), x[1] - high_bf16(a)));
                    pl[nb][1] = transpose8x8(pack_bf16(x[2] - low_bf16(b), x[3] - high_bf16(b)));
                }
            }

            // O^T += V^T P^T: rows are columns of the head.
            if constexpr (!FP8) {
                const int vrow = (lane & 7) + ((lane >> 4) << 3);
                const int vsw = vrow & 7;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t a[4];
                    ldsm4_t(a, vb + vrow * RB + (((2 * ks + ((lane >> 3) & 1)) ^ vsw) << 4));
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        mma<false>(acc[ks][nb], a[0], a[1], a[2], a[3], pb[nb][0], pb[nb][1]);
                        mma<false>(acc[ks][nb], a[0], a[1], a[2], a[3], pl[nb][0], pl[nb][1]);
                    }
                }
            } else {
                // The transposing load moves pairs of codes: lane (g, t) gets columns 2g and 2g + 1 of tokens 2t
                // and 2t + 1. The even columns become rows 0..7 of the MMA tile, the odd ones rows 8..15.
                const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
                const int vsw = CPR >= 8 ? vrow & 7 : (vrow >> 1) & 3;
#pragma unroll
                for (int c = 0; c < CPR; c += 2) {
                    uint32_t a[4];
                    ldsm4_t(a, vb + vrow * RB + (((c + (lane >> 4)) ^ vsw) << 4));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t lo = __byte_perm(a[2 * x], 0, 0x3120), hi = __byte_perm(a[2 * x + 1], 0, 0x3120);
                        const uint32_t a0 = e4m3_pair(lo), a1 = e4m3_pair(lo >> 16);
                        const uint32_t a2 = e4m3_pair(hi), a3 = e4m3_pair(hi >> 16);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma<true>(acc[c + x][nb], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
                    }
                }
            }
        }

        // ---- the warps' results of this row, joined ----
        const int64_t row_first = f0 + done - s;                     // the row's place in the list
        const bool whole = s == 0 && seg == ns;
        const int c1 = static_cast<int>(row_first / quota), c2 = static_cast<int>((row_first + ns - 1) / quota);
        const int64_t piece = static_cast<int64_t>(blockIdx.x) * 2 + (s == 0 ? 1 : 0);
        const float v_scale = FP8 && p.v_scale ? p.v_scale[h] : 1.f;
        const int d4s = p.head_dim / 4;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (nb * 8 < nh) {
                __syncthreads();                                     // part_s has been read
                float* mine_s = part_s + w * 8 * S::kPartStride;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float sum = l[nb][j];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    float* at = mine_s + (2 * t + j) * S::kPartStride;
                    if (g == 0) {
                        at[DT] = m[nb][j];
                        at[DT + 1] = sum;
                    }
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        // row g of the tile: column ks * 16 + g (FP8: 2g); row g + 8: + 8 (FP8: + 1)
                        at[ks * 16 + (FP8 ? 2 * g : g)] = acc[ks][nb][j];
                        at[ks * 16 + (FP8 ? 2 * g + 1 : g + 8)] = acc[ks][nb][j + 2];
                    }
                }
                __syncthreads();
                const int heads = min(8, nh - nb * 8);
                for (int i = tid; i < heads * d4s; i += T) {
                    const int hd = i / d4s, d = (i - hd * d4s) * 4;
                    const float* at = part_s + hd * S::kPartStride;
                    float top = kNegInf;
#pragma unroll
                    for (int k = 0; k < W; ++k) top = fmaxf(top, at[k * 8 * S::kPartStride + DT]);
                    float sum = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        const float* a = at + k * 8 * S::kPartStride;
                        const float mk = a[DT];
                        if (mk != kNegInf) {
                            const float e = exp2f(mk - top);
                            const float4 v = *reinterpret_cast<const float4*>(a + d);
                            sum += a[DT + 1] * e;
                            o.x += v.x * e;
                            o.y += v.y * e;
                            o.z += v.z * e;
                            o.w += v.w * e;
                        }
                    }
                    const int hh = nb * 8 + hd;
                    if (whole) {
                        const float inv = sum == 0.f ? 0.f : v_scale / sum;
                        *reinterpret_cast<uint2*>(p.out + row * p.out_stride + (head_at + hh) * p.head_dim + d) =
                            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                        if (p.lse && d == 0)
                            p.lse[row * p.q_heads + head_at + hh] =
                                top == kNegInf ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
                    } else {
                        *reinterpret_cast<float4*>(p.part + (piece * (NB * 8) + hh) * DT + d) = o;
                        if (d == 0)
                            *reinterpret_cast<float2*>(p.part_ml + (piece * (NB * 8) + hh) * 2) = make_float2(top, sum);
                    }
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            uint32_t* ticket = p.ticket + c1 * p.qtiles + qt;
            if (tid == 0) {
                const uint32_t old = atomicAdd(ticket, 1u);
                s_last = old == static_cast<uint32_t>(c2 - c1);
                if (s_last) *ticket = 0u;                            // zero again for the next call
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int i = tid; i < nh * d4s; i += T) {
                    const int hd = i / d4s, d = (i - hd * d4s) * 4;
                    auto piece_of = [&](int c) {
                        return ((static_cast<int64_t>(c) * p.qtiles + qt) * 2 + (c == c1 ? 1 : 0)) * (NB * 8) + hd;
                    };
                    float top = kNegInf;
                    for (int c = c1; c <= c2; ++c) top = fmaxf(top, __ldcg(p.part_ml + piece_of(c) * 2));
                    float sum = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = c1; c <= c2; ++c) {
                        const int64_t at = piece_of(c);
                        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + at * DT + d));
                        const float e = ml.x == kNegInf ? 0.f : exp2f(ml.x - top);
                        sum += ml.y * e;
                        o.x += v.x * e;
                        o.y += v.y * e;
                        o.z += v.z * e;
                        o.w += v.w * e;
                    }
                    const float inv = sum == 0.f ? 0.f : v_scale / sum;
                    *reinterpret_cast<uint2*>(p.out + row * p.out_stride + (head_at + hd) * p.head_dim + d) =
                        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                    if (p.lse && d == 0)
                        p.lse[row * p.q_heads + head_at + hd] =
                            top == kNegInf ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }

        done += seg;
        s += seg;
        if (s == ns && done < cnt) {
            s = 0;
            if (++h == p.kv_heads) {
                h = 0;
                do ++r;
                while (r < p.requests && attn_slices(p, len_of(r)) == 0);
                if (r >= p.requests) break;
            }
        }
    }
    copy_wait<0>();
}

}  // namespace gemv
