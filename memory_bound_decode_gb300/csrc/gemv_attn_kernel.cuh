// Attention of one new token per request over a paged key-value cache.
//
//   s_j = cap(scale * q . k_j),  p_j = exp(s_j - m),  out = sum_j p_j v_j / sum_j p_j
//
// over the visible tokens j of a request, with the running maximum m and sum
// of a softmax kept in FP32, so K and V are read once and no score is stored.
//
// Work split. A row is one (request, key-value head) pair; its tokens are cut
// into slices of 32 or 16. All slices of all rows form one list (request-major), and
// each CTA takes an equal, contiguous range of it, whatever the lengths are:
// the lengths live on the device, so every CTA sums them itself. Inside a CTA
// the warps take the range's slices in turn. A row inside one range is
// finished there; a row cut between CTAs leaves FP32 partial results (output,
// maximum, sum) in the workspace and the CTA that arrives last joins them in
// list order, so the result does not depend on which one that is.
//
// Tiles. The group of query heads that share a key-value head are the narrow
// side (N = 8) of the MMAs, 16 tokens of a slice (scores) or 16 columns of
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
template <int TS>   // tokens of a slice
__device__ __forceinline__ int attn_slices(const AttnParams& p, int len) {
    return len <= 0 ? 0 : (len + TS - 1) / TS - attn_begin(p, len) / TS;
}

// The slice of an instance: 32 tokens (two MMA tiles side by side hide each
// other's latency and share one reduction), 16 where two would not fit the
// registers or the ring.
template <int DT, int NB, bool FP8>
struct AttnShape {
    static constexpr int kWarps = 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSlice = (DT == 256 && !FP8) || (DT == 256 && NB == 2) || NB == 4 ? 16 : 32;
    static constexpr int kRowBytes = DT * (FP8 ? 1 : 2);
    static constexpr int kEntry = kSlice * kRowBytes;                // K or V of one slice
    static constexpr int kEntries = 196608 / (kWarps * kEntry) < 12 ? 196608 / (kWarps * kEntry) : 12;
    static constexpr int kRing = kWarps * kEntries * kEntry;
    // The warps' results meet in shared memory 8 heads and at most 128 columns at a time; behind the columns of
    // a head stand its maximum and sum.
    static constexpr int kPartCols = DT < 128 ? DT : 128;
    static constexpr int kPartStride = kPartCols + 4;
    static constexpr int kPart = kWarps * 8 * kPartStride * 4;
    // Query fragments stay in registers, or (in the same memory as kPart: they are not needed together) in shared
    // memory where the accumulators leave no registers for them.
    static constexpr bool kQueryShared = NB == 4 || (DT == 256 && NB == 2);
    static constexpr int kSmem = kRing + kPart;
    static_assert(!kQueryShared || (DT / 16) * NB * 256 <= kPart, "query fragments fit");
};

template <int DT, int NB, bool FP8>
__global__ void __launch_bounds__(AttnShape<DT, NB, FP8>::kThreads, 1)
attn_decode_kernel(const __grid_constant__ AttnParams p) {
    using S = AttnShape<DT, NB, FP8>;
    using namespace attn;
    constexpr int W = S::kWarps, T = S::kThreads, TS = S::kSlice, MT = TS / 16, E = S::kEntries;
    constexpr int RB = S::kRowBytes;
    constexpr int CPR = RB / 16;          // 16-byte chunks of a row
    constexpr int KS = DT / 16;           // MMA steps along the head
    constexpr float kNegInf = -INFINITY;
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

    extern __shared__ __align__(128) unsigned char smem[];
    float* const part_s = reinterpret_cast<float*>(smem + S::kRing);
    uint2* const q_s = reinterpret_cast<uint2*>(smem + S::kRing);
    __shared__ int32_t s_len[T];          // lengths of requests len0 .. len0 + T - 1
    __shared__ int64_t s_scan[W];
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

    // The sum of the slices, and (in the first chunk of T requests) their running sums.
    const int len_first = tid < p.requests ? attn_len(p, tid) : -1;
    const int n_first = attn_slices<TS>(p, len_first);
    s_len[tid] = len_first;
    int64_t incl = n_first;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[w] = incl;
    if (tid == 0) s_r0 = -1;
    __syncthreads();
    int64_t carry = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (i < w) incl += s_scan[i];
        carry += s_scan[i];
    }
    int64_t total = carry;
    if (p.requests > T) {
        int64_t more = 0;
        for (int r = T + tid; r < p.requests; r += T) {
            more += attn_slices<TS>(p, attn_len(p, r));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
        __syncthreads();
        if (lane == 0) s_scan[w] = more;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) total += s_scan[i];
    }

    // Requests without a visible token: zeros (nothing to average), from the CTA whose turn it is.
    for (int r = blockIdx.x; r < p.requests; r += gridDim.x) {
        if ((r < T ? s_len[r] : attn_len(p, r)) != 0) continue;
        const int64_t row = attn_row(p, r);
        uint2* o = reinterpret_cast<uint2*>(p.out + row * p.out_stride);
        for (int i = tid; i < p.q_heads * p.head_dim / 4; i += T) o[i] = make_uint2(0, 0);
        if (p.lse)
            for (int i = tid; i < p.q_heads; i += T) p.lse[row * p.q_heads + i] = kNegInf;
    }

    // This CTA's range, f0 .. f0 + cnt, of the list of slices, and the request that f0 falls in.
    total *= p.kv_heads;
    const int64_t quota = max((total + ctas - 1) / ctas, static_cast<int64_t>(p.min_slices));
    const int64_t f0 = cta * quota;
    if (f0 >= total) return;
    const int cnt = static_cast<int>(min(quota, total - f0));
    auto claim = [&](int r, int n, int64_t end) {                    // `end`: slices up to request r, a head
        const int64_t lo = (end - n) * p.kv_heads;
        if (lo <= f0 && f0 < end * p.kv_heads) {
            s_r0 = r;
            s_off = f0 - lo;
        }
    };
    claim(tid, n_first, incl);
    int len0 = 0;
    for (int base = T; base < p.requests && carry * p.kv_heads <= f0; base += T) {   // the same for all threads
        const int len = base + tid < p.requests ? attn_len(p, base + tid) : -1;
        const int n = attn_slices<TS>(p, len);
        incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();                                            // s_scan and s_len have been read
        if (lane == 31) s_scan[w] = incl;
        s_len[tid] = len;
        len0 = base;
        __syncthreads();
        int64_t before = carry;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < w) before += s_scan[i];
            carry += s_scan[i];
        }
        claim(base + tid, n, before + incl);
    }
    __syncthreads();
    const int r0 = s_r0;
    if (r0 < 0) return;                                             // only if lens changed under the call
    auto len_of = [&](int r) { return r - len0 < T ? s_len[r - len0] : attn_len(p, r); };

    const int ns0 = max(1, attn_slices<TS>(p, len_of(r0)));
    const int h_first = s_off >> 31 ? static_cast<int>(s_off / ns0) : static_cast<int>(s_off) / ns0;
    const int s_first = static_cast<int>(s_off - static_cast<int64_t>(h_first) * ns0);

    // ---- copies of K and V into this warp's ring: entries K0 V0 K1 V1 ..., E of them at a time ----
    const uint32_t ring = sm_addr(smem) + static_cast<uint32_t>(w) * E * S::kEntry;
    const int warp_slices = cnt > w ? (cnt - w + W - 1) / W : 0;
    const int chunks = p.head_dim * (FP8 ? 1 : 2) / 16;
    int pr = r0, ph = h_first, ps = s_first, pns = ns0, plen = len_of(r0);
    int issued = 0;                       // entries
    uint32_t valid_of = 0;                // lane i: the visible tokens of slice i (modulo 32)
    int next_page = -1, next_in = -1;     // lane i: page and place of token i of the next slice
    int next_h = 0;
    int64_t off = -1;                     // lane i: byte offset of token i of the slice whose K went out last
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
                    pns = attn_slices<TS>(p, plen);
                } while (pns == 0);
            }
        }
        const int begin = attn_begin(p, plen);
        const int tok = (begin / TS + ps) * TS + (lane & (TS - 1));
        const bool in = tok >= begin && tok < plen;
        const int blk = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
        next_in = in ? tok - blk * p.page_size : -1;
        next_page = in ? p.table[pr * p.table_stride + blk] : -1;
        next_h = ph;
    };
    auto copy_rows = [&](const unsigned char* base, uint32_t dst0) {
#pragma unroll
        for (int i = 0; i < TS * CPR / 32; ++i) {
            const int idx = i * 32 + lane, row = idx / CPR, ch = idx % CPR;
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            const int sw = CPR >= 8 ? row & 7 : (row >> 1) & 3;
            const int n = o >= 0 && ch < chunks ? 16 : 0;            // 0: the chunk is filled with zeros
            copy16(dst0 + row * RB + ((ch ^ sw) << 4), base + (n ? o + ch * 16 : 0), n);
        }
    };
    auto issue = [&]() {
        const int slice = issued >> 1;
        if (slice < warp_slices) {
            const uint32_t dst = ring + (issued % E) * S::kEntry;
            if ((issued & 1) == 0) {
                off = -1;
                if (next_in >= 0) {
                    if (next_page >= 0 && next_page < p.num_pages)
                        off = next_page * p.page_stride + next_h * p.head_stride + next_in * p.slot_stride;
                    else
                        atomicOr(&g_attn_status, kStatusBadPage);
                }
                const uint32_t valid = __ballot_sync(0xffffffffu, off >= 0);
                if (lane == (slice & 31)) valid_of = valid;
                copy_rows(p.kc, dst);
                if (slice + 1 < warp_slices) settle(W);
            } else {
                copy_rows(p.vc, dst);
            }
        }
        ++issued;
        copy_commit();
    };
    if (warp_slices > 0) settle(w);
#pragma unroll 1
    for (int i = 0; i < E; ++i) issue();

    // ---- rows of the range, one after the other ----
    int r = r0, h = h_first, s = s_first, done = 0, li = w, taken = 0;   // taken: entries
    while (done < cnt) {
        const int len = len_of(r);
        const int ns = attn_slices<TS>(p, len);
        const int seg = min(ns - s, cnt - done);
        if (seg <= 0) break;
        const int64_t row = attn_row(p, r);
        const int64_t head_at = static_cast<int64_t>(h) * p.group + head0;

        // Query fragments (B operand: 16 columns of the head x 8 heads).
        uint32_t qf[S::kQueryShared ? 1 : KS][S::kQueryShared ? 1 : NB][2];
        float col_scale[NB][2];
        auto load_query = [&](int nb, int ks, uint32_t (&f)[2]) {
            const bool in = nb * 8 + g < nh;
            const uint16_t* qp = p.q + row * p.q_stride + (head_at + nb * 8 + g) * p.head_dim;
            if constexpr (!FP8) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int d = ks * 16 + b * 8 + 2 * t;
                    f[b] = in && d < p.head_dim ? *reinterpret_cast<const uint32_t*>(qp + d) : 0u;
                }
            } else {
                const int d = ks * 16 + 4 * t;
                const uint2 v = in && d < p.head_dim ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
                f[0] = v.x;
                f[1] = v.y;
            }
        };
        if constexpr (S::kQueryShared) __syncthreads();              // part_s has been read
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            uint32_t f[KS][2];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) load_query(nb, ks, f[ks]);
            if constexpr (!FP8) {
                col_scale[nb][0] = col_scale[nb][1] = p.scale;
            } else {
                // The FP8 cache is widened to FP16 (exact); q is brought to FP16 by a power of two per head
                // that puts its largest value in [1, 2): what that loses is below 2^-24 of that value.
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        top = fmaxf(top, fmaxf(fabsf(low_bf16(f[ks][b])), fabsf(high_bf16(f[ks][b]))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
                e = top > 0.f ? max(-126, min(126, e)) : 0;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        f[ks][b] = pack_f16(low_bf16(f[ks][b]) * down, high_bf16(f[ks][b]) * down);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                const float ksc = p.scale * (p.k_scale ? p.k_scale[h] : 1.f);
                col_scale[nb][0] = __shfl_sync(0xffffffffu, up, 8 * t) * ksc;
                col_scale[nb][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4) * ksc;
            }
            if constexpr (S::kQueryShared) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    if (ks % W == w) q_s[(nb * KS + ks) * 32 + lane] = make_uint2(f[ks][0], f[ks][1]);
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qf[ks][nb][0] = f[ks][0];
                    qf[ks][nb][1] = f[ks][1];
                }
            }
        }
        if constexpr (S::kQueryShared) __syncthreads();
        auto query = [&](int ks, int nb) {
            if constexpr (S::kQueryShared) return q_s[(nb * KS + ks) * 32 + lane];
            else return make_uint2(qf[ks][nb][0], qf[ks][nb][1]);
        };

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
            copy_wait<E - 1>();
            __syncwarp();
            const uint32_t valid = __shfl_sync(0xffffffffu, valid_of, (taken >> 1) & 31);

            // S^T = K Q^T: rows g and g + 8 of a tile are tokens, columns 2t and 2t + 1 heads.
            float sc[MT][NB][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) sc[mt][nb][0] = sc[mt][nb][1] = sc[mt][nb][2] = sc[mt][nb][3] = 0.f;
            {
                const uint32_t kb = ring + (taken % E) * S::kEntry;
                const int arow = lane & 15;
                const int asw = CPR >= 8 ? arow & 7 : (arow >> 1) & 3;
#pragma unroll
                for (int c = 0; c < CPR; c += 2) {                   // two 16-byte chunks of the rows
                    uint32_t a[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        ldsm4(a[mt], kb + (mt * 16 + arow) * RB + (((c + (lane >> 4)) ^ asw) << 4));
                    if constexpr (!FP8) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const uint2 b = query(c / 2, nb);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma<false>(sc[mt][nb], a[mt][0], a[mt][1], a[mt][2], a[mt][3], b.x, b.y);
                        }
                    } else {
                        // Bytes 4t .. 4t + 3 of a chunk: columns 2t, 2t + 1 and 2t + 8, 2t + 9 of the step, by a
                        // permutation of the chunk's columns that q's fragments share.
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t f[MT][4];
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                f[mt][0] = e4m3_pair(a[mt][2 * x]);
                                f[mt][1] = e4m3_pair(a[mt][2 * x + 1]);
                                f[mt][2] = e4m3_pair(a[mt][2 * x] >> 16);
                                f[mt][3] = e4m3_pair(a[mt][2 * x + 1] >> 16);
                            }
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                const uint2 b = query(c + x, nb);
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
                                    mma<true>(sc[mt][nb], f[mt][0], f[mt][1], f[mt][2], f[mt][3], b.x, b.y);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            ++taken;
            issue();                                                 // into the entry just read

            // Running maximum and sum, in powers of two.
            uint32_t pb[MT][NB][2], pl[FP8 ? 1 : MT][FP8 ? 1 : NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float x[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float v = sc[mt][nb][j] * col_scale[nb][j & 1];
                        if (p.softcap > 0.f) v = p.softcap * tanhf(v / p.softcap);
                        v *= kLog2e;
                        x[mt][j] = valid >> (mt * 16 + g + (j & 2) * 4) & 1u ? v : kNegInf;
                    }
                float corr[2], base[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(x[0][j], x[0][j + 2]);
                    if constexpr (MT == 2) top = fmaxf(top, fmaxf(x[1][j], x[1][j + 2]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[nb][j]);
                    base[j] = top == kNegInf ? 0.f : top;
                    corr[j] = exp2f(m[nb][j] - base[j]);
                    m[nb][j] = top;
                }
                l[nb][0] *= corr[0];
                l[nb][1] *= corr[1];
                if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        acc[ks][nb][0] *= corr[0];
                        acc[ks][nb][1] *= corr[1];
                        acc[ks][nb][2] *= corr[0];
                        acc[ks][nb][3] *= corr[1];
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[mt][j] = exp2f(x[mt][j] - base[j & 1]);
                    l[nb][0] += x[mt][0] + x[mt][2];
                    l[nb][1] += x[mt][1] + x[mt][3];
                    // P as the B operand. FP16 beside an FP8 cache (2^-12 relative). Beside a BF16 cache P has to
                    // be BF16, whose 2^-9 would double the rounding error of a BF16 output: it goes in two parts
                    // (the rest in a second BF16), 2^-18 together.
                    if constexpr (FP8) {
                        pb[mt][nb][0] = transpose8x8(pack_f16(x[mt][0], x[mt][1]));
                        pb[mt][nb][1] = transpose8x8(pack_f16(x[mt][2], x[mt][3]));
                    } else {
                        const uint32_t a = pack_bf16(x[mt][0], x[mt][1]), b = pack_bf16(x[mt][2], x[mt][3]);
                        pb[mt][nb][0] = transpose8x8(a);
                        pb[mt][nb][1] = transpose8x8(b);
                        pl[mt][nb][0] = transpose8x8(pack_bf16(x[mt][0] - low_bf16(a), x[mt][1] - high_bf16(a)));
                        pl[mt][nb][1] = transpose8x8(pack_bf16(x[mt][2] - low_bf16(b), x[mt][3] - high_bf16(b)));
                    }
                }
            }

            // O^T += V^T P^T: rows are columns of the head.
            copy_wait<E - 1>();
            __syncwarp();
            const uint32_t vb = ring + (taken % E) * S::kEntry;
            if constexpr (!FP8) {
                const int vrow = (lane & 7) + ((lane >> 4) << 3);
                const int vsw = vrow & 7;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        ldsm4_t(a, vb + (mt * 16 + vrow) * RB + (((2 * ks + ((lane >> 3) & 1)) ^ vsw) << 4));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            mma<false>(acc[ks][nb], a[0], a[1], a[2], a[3], pb[mt][nb][0], pb[mt][nb][1]);
                            mma<false>(acc[ks][nb], a[0], a[1], a[2], a[3], pl[mt][nb][0], pl[mt][nb][1]);
                        }
                    }
            } else {
                // The transposing load moves pairs of codes: lane (g, t) gets columns 2g and 2g + 1 of tokens 2t
                // and 2t + 1. The even columns become rows 0..7 of the MMA tile, the odd ones rows 8..15.
                const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
                const int vsw = CPR >= 8 ? vrow & 7 : (vrow >> 1) & 3;
#pragma unroll
                for (int c = 0; c < CPR; c += 2)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        ldsm4_t(a, vb + (mt * 16 + vrow) * RB + (((c + (lane >> 4)) ^ vsw) << 4));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t lo = __byte_perm(a[2 * x], 0, 0x3120);
                            const uint32_t hi = __byte_perm(a[2 * x + 1], 0, 0x3120);
                            const uint32_t a0 = e4m3_pair(lo), a1 = e4m3_pair(lo >> 16);
                            const uint32_t a2 = e4m3_pair(hi), a3 = e4m3_pair(hi >> 16);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma<true>(acc[c + x][nb], a0, a1, a2, a3, pb[mt][nb][0], pb[mt][nb][1]);
                        }
                    }
            }
            __syncwarp();
            ++taken;
            issue();
        }

        // ---- the warps' results of this row, joined ----
        const bool whole = s == 0 && seg == ns;
        const int64_t piece = static_cast<int64_t>(blockIdx.x) * 2 + (s == 0 ? 1 : 0);
        const float v_scale = FP8 && p.v_scale ? p.v_scale[h] : 1.f;
        auto store = [&](int hd, int d, float4 o, float top, float sum) {
            const float inv = sum == 0.f ? 0.f : v_scale / sum;
            *reinterpret_cast<uint2*>(p.out + row * p.out_stride + (head_at + hd) * p.head_dim + d) =
                make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            if (p.lse && d == 0)
                p.lse[row * p.q_heads + head_at + hd] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
        };
        constexpr int KP = S::kPartCols / 16;                        // steps of a round
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float sums[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sums[j] = l[nb][j];
                sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], 4);
                sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], 8);
                sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], 16);
            }
            const int heads = min(8, nh - nb * 8);
#pragma unroll
            for (int d0 = 0; d0 < DT; d0 += S::kPartCols) {
                if (heads <= 0 || d0 >= p.head_dim) continue;
                __syncthreads();                                     // part_s (or q_s) has been read
                float* mine_s = part_s + w * 8 * S::kPartStride;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (2 * t + j < heads) {
                        float* at = mine_s + (2 * t + j) * S::kPartStride;
                        if (g == 0) {
                            at[S::kPartCols] = m[nb][j];
                            at[S::kPartCols + 1] = sums[j];
                        }
#pragma unroll
                        for (int k = 0; k < KP; ++k) {
                            // row g of the tile: column k * 16 + g (FP8: 2g); row g + 8: + 8 (FP8: + 1)
                            at[k * 16 + (FP8 ? 2 * g : g)] = acc[d0 / 16 + k][nb][j];
                            at[k * 16 + (FP8 ? 2 * g + 1 : g + 8)] = acc[d0 / 16 + k][nb][j + 2];
                        }
                    }
                }
                __syncthreads();
                const int d4s = min(S::kPartCols, p.head_dim - d0) / 4;
                for (int i = tid; i < heads * d4s; i += T) {
                    const int hd = i / d4s, d = (i - hd * d4s) * 4;
                    const float* at = part_s + hd * S::kPartStride;
                    float mk[W], top = kNegInf;
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        mk[k] = at[k * 8 * S::kPartStride + S::kPartCols];
                        top = fmaxf(top, mk[k]);
                    }
                    float sum = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        const float* a = at + k * 8 * S::kPartStride;
                        if (mk[k] != kNegInf) {
                            const float e = exp2f(mk[k] - top);
                            const float4 v = *reinterpret_cast<const float4*>(a + d);
                            sum += a[S::kPartCols + 1] * e;
                            o.x += v.x * e;
                            o.y += v.y * e;
                            o.z += v.z * e;
                            o.w += v.w * e;
                        }
                    }
                    const int hh = nb * 8 + hd;
                    if (whole) {
                        store(hh, d0 + d, o, top, sum);
                    } else {
                        *reinterpret_cast<float4*>(p.part + (piece * (NB * 8) + hh) * DT + d0 + d) = o;
                        if (d0 + d == 0)
                            *reinterpret_cast<float2*>(p.part_ml + (piece * (NB * 8) + hh) * 2) = make_float2(top, sum);
                    }
                }
            }
        }
        if (!whole) {
            const int64_t row_first = f0 + done - s;                 // the row's place in the list
            const int c1 = static_cast<int>(row_first / quota), c2 = static_cast<int>((row_first + ns - 1) / quota);
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
                const int d4s = p.head_dim / 4;
                for (int i = tid; i < nh * d4s; i += T) {
                    const int hd = i / d4s, d = (i - hd * d4s) * 4;
                    auto piece_of = [&](int c) {
                        return ((static_cast<int64_t>(c) * p.qtiles + qt) * 2 + (c == c1 ? 1 : 0)) * (NB * 8) + hd;
                    };
                    float top = kNegInf;
#pragma unroll 4
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
                    store(hd, d, o, top, sum);
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
                while (r < p.requests && attn_slices<TS>(p, len_of(r)) == 0);
                if (r >= p.requests) break;
            }
        }
    }
    copy_wait<0>();
}

}  // namespace gemv
