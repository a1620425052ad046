// Attention of one new token per request over a paged key-value cache.
//
//   s_j = cap(scale * q . k_j),  p_j = exp(s_j - m),  out = sum_j p_j v_j / sum_j p_j
//
// over the visible tokens j of a request, with the running maximum m and sum
// of a softmax kept in FP32, so K and V are read once and no score is stored.
//
// Work split. A row is one (request, key-value head) pair; its tokens are cut
// into slices of 16, 32 or 64. All slices of all rows form one list
// (request-major); each CTA takes an equal, contiguous range of it, and each
// warp an equal, contiguous part of that, whatever the lengths are: the lengths
// live on the device, so every CTA sums them itself. (Teams of up to 8 CTAs
// take the same range for a head each of a block of heads.) A warp works through its
// part alone, row after row, without a barrier of the CTA: rows of a few
// hundred tokens cost no more than their bytes. A row inside one warp's part
// is finished there. Of the others each warp has two pieces at most, its first
// and its last; the CTA joins its warps' pieces once, at the end, and a row
// cut between CTAs is joined by the CTA that arrives last, through the
// workspace. Pieces (FP32 output, maximum, sum) are always joined in list
// order, so the result does not depend on which CTA that is.
//
// Scales. An FP8 cache with one scale per head has it in q and in the output's
// factor. With a scale ks, vs for each block of tokens, a score is multiplied by
// its token's ks, and with M the running maximum of s_j + log vs_j
//
//   p_j = exp(s_j - M),  out = sum_j (p_j vs_j) code_j / sum_j p_j:
//
// one exponential and one maximum as before, and the weights p_j vs_j, which
// meet the codes in FP16, are relative to the largest of the products that are
// summed, however far the scales of the blocks are apart. (The logarithm of vs
// is in M alone, so its error divides out.) The sum of the p_j needs more of
// FP32's range than the weights: with vs from 2^-60 to 2^128 the largest p_j is
// between 2^-128 and 2^60 of a maximum of 1. So p_j is kept times 2^20 more
// than the weights (2^31 tokens of 2^60 end below 2^127; what is lost is below
// 2^-33 of the largest p_j, 2^-41 where scales are at most 2^120), and a sum
// moves to another maximum by the root of the factor, twice: the factor may be
// below 2^-126 where the product is not. The scales of a slice's tokens come by
// asynchronous copies beside its K, counted on the same barrier.
//
// Tiles. The group of query heads that share a key-value head are the narrow
// side (N = 8) of the MMAs, 16 tokens of a slice (scores) or 16 columns of
// the head (output) the wide one: S^T = K Q^T and O^T = V^T P^T. K and V then
// come straight from shared memory as the A operand (ldmatrix, transposed for
// V), each fetched once, and the running maximum and sum of a head sit in the
// same lanes as its output columns. S^T becomes the B operand of the second
// product by an 8x8 transposition in registers (movmatrix). These are the
// warp-level MMAs: with 4 heads on a key-value head a byte of K or V takes 4
// operations, and the tensor pipe is 13-23% busy while the HBM is the limit.
//
// What bounds it. Long lists the HBM: 64 requests of 16,384 to 32,768 tokens of
// 8 heads of 128 (BF16, 6.44 GB) 885 us, 7.3 TB/s, 1.07 of a copy's rate; FP8,
// 32 requests of up to 16,384 85 us, 6.3 TB/s. Groups of 16 heads of 256
// columns the warps' instructions (64 us for 46 us of bytes). Short ones
// latency: 1 x 1,000 tokens 8.8 us, of which the launch, the lengths, the page
// numbers and the first tokens follow each other for 5, and the pieces' join
// takes 3.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "gemv_attn_internal.h"
#include "gemv_common.cuh"

namespace gemv {

static __device__ unsigned int g_attn_status;
constexpr unsigned int kStatusBadPage = 2u;   // kStatusWaitTimeout (1) too

#ifdef GEMV_DEBUG_DROP_X
constexpr bool kDrop = true;     // the test build whose waits are meant to run out: instances with tensor copies never
                                 // copy V, the others never count their queries in
#else
constexpr bool kDrop = false;
#endif

namespace attn {

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4_or_zero(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// This thread's arrival at the barrier, once its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
// A tensor copy's description is fetched on its first use, unless asked for before.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }
// How the L2 is to keep what a copy brings.
__device__ __forceinline__ uint64_t keep_first_out() {
    uint64_t r;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
    return r;
}
__device__ __forceinline__ uint64_t keep_normal() {
    uint64_t r;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(r));
    return r;
}
// One box of the pool's 4-D view (column, slot, head, page).
__device__ __forceinline__ void copy_box(uint32_t dst, const void* map, int col, int slot, int head, int page,
                                         uint32_t bar, uint64_t keep) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;"
                 :: "r"(dst), "l"(map), "r"(col), "r"(slot), "r"(head), "r"(page), "r"(bar), "l"(keep) : "memory");
}
// Wait for the barrier's phase, for at most kMbarWaitLimit rounds; false (and the status bit) if they ran out.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < kMbarWaitLimit; ++i) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred P1;\n\tmbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
                     "selp.b32 %0, 1, 0, P1;\n\t}" : "=r"(done) : "r"(bar), "r"(parity) : "memory");
        if (done) return true;
    }
    atomicOr(&g_attn_status, kStatusWaitTimeout);
    return false;
}

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

// Four E4M3 codes to FP16, exactly: the low two to lo, the high two to hi.
__device__ __forceinline__ void e4m3_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(v));
}
// 2^x; below 2^-126: 0.
__device__ __forceinline__ float exp2_ftz(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float log2_ftz(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {   // towards zero
    uint32_t r;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// What scores are taken relative to: their maximum, or 0 where it is infinite (inf - inf would be NaN; so a score of
// +inf has the weight inf, the sum is inf as it should be, and the outputs are inf / inf).
__device__ __forceinline__ float base_of(float top) { return fabsf(top) == INFINITY ? 0.f : top; }
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace attn

__device__ __forceinline__ int attn_cut(const AttnParams& p, int len) {   // to what a row of the table holds
    if (len <= p.max_len) return len;
    atomicOr(&g_attn_status, kStatusBadPage);
    return p.max_len;
}
// Tokens of request r that its query can reach: its length, cut to what its
// row of the table holds (with a status bit); 0 for an empty or a refused
// request, negative for one that has no query row in this call.
static __device__ __noinline__ int attn_len(const AttnParams& p, int r) {
    const int len = p.lens[r];
    const bool refused = p.status && p.status[r] != 0;
    if (p.token_start) {
        const int a = p.token_start[r], b = p.token_start[r + 1];
        if (b <= a) return -1;
        if (a < 0 || b > p.rows) {
            if (!refused) atomicOr(&g_attn_status, kStatusBadPage);
            return -1;
        }
    }
    return refused ? 0 : attn_cut(p, len);
}
__device__ __forceinline__ int attn_row(const AttnParams& p, int r) {
    return p.token_start ? p.token_start[r + 1] - 1 : r;
}
__device__ __forceinline__ int attn_begin(const AttnParams& p, int len) {
    return p.window > 0 && len > p.window ? len - p.window : 0;
}
template <int TS>   // tokens of a slice
__device__ __forceinline__ int attn_slices(const AttnParams& p, int len) {
    return len <= 0 ? 0 : (len + TS - 1) / TS - attn_begin(p, len) / TS;
}

// DT: head size of the instance (head_dim <= DT; columns past head_dim are
// zero). NB: blocks of 8 query heads. BLOCK: FP8 with a scale for each block of
// tokens and head.
template <int DT, int NB, bool FP8, bool TMA, bool BLOCK = false>
struct AttnShape {
    static_assert(FP8 || !BLOCK, "codes have scales");
    static constexpr int kWarps = kAttnWarps;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSlice = attn_slice(DT, NB, FP8, TMA, BLOCK);
    static constexpr int kRowBytes = DT * (FP8 ? 1 : 2);
    static constexpr int kEntry = kSlice * kRowBytes;                // K or V of one slice
    static constexpr int kEntries = kAttnRing / kEntry < 8 ? kAttnRing / kEntry : 8;
    static constexpr int kRing = kWarps * kAttnRing;
    static_assert(kEntry % 1024 == 0, "entries start where the swizzle's pattern does");
    // A warp's last piece takes the place of its ring when that is empty.
    static_assert(NB * 8 * DT * 4 <= kAttnRing, "a piece fits the ring");
    // Query fragments stay in registers where the accumulators leave room for them; else the products read them
    // from shared memory each time. Either way a warp keeps the queries of a row there as they come, heads apart in
    // banks (32-bit reads of BF16, 64-bit ones of FP16).
    static constexpr bool kQueryShared = NB == 4 || (DT == 256 && NB == 2);
    static constexpr int kRawStride = DT * 2 + (FP8 ? 32 : 16);
    static constexpr int kRaw = NB * 8 * kRawStride;
    // A warp's first piece waits in shared memory for the others where there is room, else in the workspace.
    static constexpr int kFirst = NB * 8 * DT * 4;
    // Scales of k and of v of the tokens of the slices in flight, a place beside each entry of K (and read before the
    // entry's next copy goes out).
    static constexpr int kScalePlaces = kEntries / 2;
    static constexpr int kScales = BLOCK ? kScalePlaces * kSlice * 8 : 0;
    static_assert(kScalePlaces >= 1 && (kEntries & (kEntries - 1)) == 0, "entries are K and V in turn");
    static constexpr bool kFirstShared = kRing + kWarps * (kRaw + kScales + kFirst) + 8192 <= 232448;
    static constexpr int kScalesAt = kRing + kWarps * (kRaw + (kFirstShared ? kFirst : 0));
    static constexpr int kSmem = kScalesAt + kWarps * kScales;
    static_assert(kSmem + 8192 <= 232448, "shared memory");
};

template <int DT, int NB, bool FP8, bool TMA, bool BLOCK = false>
__global__ void __launch_bounds__(AttnShape<DT, NB, FP8, TMA, BLOCK>::kThreads, 1)
attn_decode_kernel(const __grid_constant__ AttnParams p) {
    using S = AttnShape<DT, NB, FP8, TMA, BLOCK>;
    using namespace attn;
    constexpr int W = S::kWarps, T = S::kThreads, TS = S::kSlice, MT = TS / 16, E = S::kEntries;
    constexpr int RB = S::kRowBytes;
    constexpr int CPR = RB / 16;          // 16-byte chunks of a row
    constexpr int KS = DT / 16;           // MMA steps along the head
    constexpr int H = NB * 8;             // query heads of a piece
    constexpr float kNegInf = -INFINITY;
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
    // Weights that meet V as FP16 are kept times 2^15 (the largest is 1): below 2^-14 FP16 has fewer bits.
    constexpr float kUp = FP8 ? 15.f : 0.f;
    // A sum without the scales of v, which those of blocks are not in, is kept times 2^20 more.
    constexpr float kSumUp = BLOCK ? kUp + 20.f : kUp, kSumDown = BLOCK ? 0x1p-35f : FP8 ? 0x1p-15f : 1.f;
    // Such a sum where the maximum moves: times 2^d (e: 2^d itself, which may be too small for FP32 where the product is not).
    auto moved = [](float sum, float d, float e) {
        if constexpr (!BLOCK) return sum * e;
        const float root = exp2_ftz(0.5f * d);
        return sum * root * root;
    };

    // A piece of a row: slices s .. s + seg - 1 of ns, the first of them slice `at` of the CTA's range.
    struct Piece {
        int valid, r, h, s, seg, ns, at;
        int row;                          // of q and out
        float v_scale;
    };
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t s_bar[W * E];     // one per ring entry: its copies have landed
    __shared__ uint64_t s_qbar[W];        // the same for a warp's queries
    __shared__ Piece s_piece[2 * W];      // each warp's first and last
    __shared__ float2 s_ml[2 * W][H];     // their maxima and sums
    __shared__ int32_t s_len[T];          // lengths of requests len0 .. len0 + T - 1
    __shared__ int2 s_scan[W];
    __shared__ int32_t s_off[W];
    __shared__ float s_scales[W][2];      // FP8: scales of k and v of the row that q_raw holds
    __shared__ int32_t s_req[W];
    __shared__ int32_t s_last[2];

    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    // Integer divisions take long (0.05 us each, where everything waits for them): few are left.
    const int unit = p.qtiles == 1 ? blockIdx.x : blockIdx.x / p.qtiles;
    const int qt = blockIdx.x - unit * p.qtiles;
    // CTAs work in teams of 2, 4 or 8 where the KV heads divide into such blocks: the list is one of head blocks, and
    // each CTA of a team takes its own head of the block. They read neighbouring memory at the same time, and the HBM
    // gives more for it (FP8, 32 x 16,384 tokens: 220 -> 167 us; BF16, 64 x 16,384 to 32,768:
    // 927 -> 884).
    const int blocks = p.kv_heads >> p.team_shift;
    const int cta = unit >> p.team_shift, member = unit & ((1 << p.team_shift) - 1);
    auto head_of = [&](int block) { return (block << p.team_shift) + member; };
    // The place in the grid of this team's CTA c (of this one's head).
    auto place_of = [&](int c) { return ((c << p.team_shift) + member) * p.qtiles + qt; };
    const int head0 = qt * H;                                        // first query head of the group
    const int nh = min(H, p.group - head0);                          // query heads of this tile
    unsigned char* const ring_p = smem + w * kAttnRing;
    unsigned char* const q_raw = smem + S::kRing + w * S::kRaw;

    pdl_launch_dependents();
    if (lane == 0) {
        // A tensor copy counts its bytes (one arrival arms the barrier), per-thread copies arrive for each lane.
        for (int i = 0; i < E; ++i) mbar_init(&s_bar[w * E + i], !TMA ? 32 : BLOCK && i % 2 == 0 ? 33 : 1);
        mbar_init(&s_qbar[w], 32);
        fence_mbar_init_cluster();
        s_req[w] = -1;
        s_scales[w][0] = s_scales[w][1] = 1.f;
        s_piece[2 * w].valid = s_piece[2 * w + 1].valid = 0;
    }
    for (int i = lane; i < S::kRaw / 16; i += 32) reinterpret_cast<uint4*>(q_raw)[i] = make_uint4(0, 0, 0, 0);
    // The table into the L2, a line per thread of the grid (no matter who writes it before this call): a page number
    // is needed as soon as the lengths are known. The lengths too, and the tensor copies' descriptions (0.2 us).
    const int64_t line = (static_cast<int64_t>(blockIdx.x) * T + tid) * 32;
    if (line < p.table_entries) prefetch_l2(p.table + line);
    if (tid * 32 < p.requests) prefetch_l2(p.lens + tid * 32);
    if (TMA && lane == 0 && w < 2) prefetch_map(w == 0 ? &p.kmap : &p.vmap);
    __syncwarp();
    pdl_wait_prerequisites();

    // ---- the sum of the slices, and (in the first chunk of requests) their running sums ----
    // Up to 32 requests each warp sums up for itself, with its copy of the lengths and no barrier (0.5 us less of
    // every call; 1 x 1,000 tokens 10.7 -> 10.2).
    const bool few = p.requests <= 32;
    const int copy = few ? w * 32 : 0, first_of = tid - copy;        // this thread's request of the first chunk
    const int len_first = first_of >= p.requests      ? -1
                          : p.token_start || p.status ? attn_len(p, first_of)
                                                      : attn_cut(p, p.lens[first_of]);
    const int n_first = attn_slices<TS>(p, len_first);
    s_len[tid] = len_first;
    int incl = n_first;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    int longest = __reduce_max_sync(0xffffffffu, n_first);
    int carry = 0;
    if (few) {
        carry = __shfl_sync(0xffffffffu, incl, 31);
        __syncwarp();                                                // s_len is written
    } else {
        if (lane == 31) s_scan[w] = make_int2(incl, longest);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int2 of = s_scan[i];
            if (i < w) incl += of.x;
            carry += of.x;
            longest = max(longest, of.y);
        }
    }
    int total = carry;
    if (p.requests > T) {
        int more = 0;
#pragma unroll 1
        for (int r = T + tid; r < p.requests; r += T) more += attn_slices<TS>(p, attn_len(p, r));
        more = __reduce_add_sync(0xffffffffu, more);
        __syncthreads();
        if (lane == 0) s_scan[w].x = more;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) total += s_scan[i].x;
    }

    // Requests without a visible token, or refused: zeros (nothing to average), from the CTA whose turn it is.
    for (int r = blockIdx.x; r < p.requests; r += gridDim.x) {
        if ((r < T ? s_len[copy + r] : attn_len(p, r)) != 0) continue;
        const int row = attn_row(p, r);
        uint2* o = reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(row) * p.out_stride);
        for (int i = tid; i < p.q_heads * p.head_dim / 4; i += T) o[i] = make_uint2(0, 0);
        if (p.lse)
            for (int i = tid; i < p.q_heads; i += T) p.lse[static_cast<int64_t>(row) * p.q_heads + i] = kNegInf;
    }

    // ---- the CTA's range f0 .. f0 + cnt of the list, this warp's part of it, and the requests the parts begin in ----
    const bool alike = p.requests <= T && static_cast<int64_t>(longest) * p.requests == total;   // (one request, say)
    total *= blocks;                                                 // below 2^31: checked by the host
    // At least a slice per warp. Rows of up to two per warp are better not cut between CTAs, and of up to four if
    // that leaves work for a quarter of the CTAs: the slices of a warp come 1.3 us after each other, a join across
    // CTAs takes 3 to 4 (measured before later steps: 8 x 1,000 tokens uncut 12.6 us, cut 14.4; 1 x 1,000 uncut 11.9,
    // cut 10.3).
    const uint64_t short_of = max(total - 1, 0);
    // total / teams, rounded up
    const int even = static_cast<int>(p.cta_part ? __umul64hi(short_of, p.cta_part) : short_of) + 1;
    // With a scale for each block a CTA takes the rows of up to two slices per warp that begin in its range, whole, and
    // longer ones are cut evenly (us, ranges that cut rows of any length -> so: 16 requests of 0 to 128 tokens
    // 10.6 -> 7.8, to 1,024 14.6 -> 12.0, to 2,048 19.5 -> 15.8, 13 of 1 to 2,000 20.1 -> 15.2; whole rows of up to four
    // slices per warp 17.5 and 16.1 in the last two). With more requests than threads rows are cut as they come; ranges
    // long enough to cut few of them, as for the other kinds, took as long (400 requests of 0 to 64 tokens 21.9 and 22.0,
    // to 300 41.4 and 41.5, to 1,024 82.6 and 82.6). Rows of one length go by the rule below, whole or cut: 8 KV heads,
    // cut -> whole, 1 x 1,000 9.4 -> 9.9, 2 9.8 -> 10.0, 8 10.3 -> 10.2; 2 x 600 9.7 -> 9.6, 4 10.0 -> 9.8, 8 10.2 -> 9.9.
    const bool whole_rows = BLOCK && longest <= 2 * W && p.requests <= T;
    const bool uncut = !BLOCK && (longest <= 2 * W || (longest <= 4 * W && even * 4 >= longest));
    int quota = whole_rows ? even : max(even, max(W, uncut ? longest : 0));
    // Rows of one length go to CTAs of their own where that adds no more than a slice per warp (a CTA between two rows
    // may be the last of both and join them one after the other: 1 x 8,000 tokens 17.7 us, so 15.0), or where a warp
    // has up to 16 slices (a join less: 13 x 2,000 tokens 26.0 -> 22.6 us, 16 x 4,000 48.0 -> 44.4; but 10 x 4,000
    // 34.2 -> 35.8).
    int per_row = 0, f0 = 0, row_end = total;                        // CTAs of a row, or 0
    int first_of_row = 0;                                            // its first CTA
    if (alike && !uncut && total > 0 && p.row_ctas > 0) {
        const int q = max(W, (longest + p.row_ctas - 1) / p.row_ctas);
        if (q <= max(quota + W, 16 * W)) {
            quota = q;
            per_row = (longest + q - 1) / q;
            if (cta >= p.requests * blocks * per_row) return;
            const int row = cta < per_row ? 0 : cta / per_row;
            first_of_row = row * per_row;
            f0 = row * longest + (cta - first_of_row) * q;
            row_end = (row + 1) * longest;
        }
    }
    if (per_row == 0) f0 = cta * quota;                              // below total + grid * quota
    if (f0 >= total) return;
    int cnt = min(quota, row_end - f0);
    if constexpr (BLOCK) {
        if (whole_rows && per_row == 0) {
            const int first = (incl - n_first) * blocks, last = incl * blocks;   // of this thread's request: its rows
            auto next_row = [&](int x) { return first + (x - first + n_first - 1) / n_first * n_first; };
            const int f1 = f0 + cnt;
            if (few) {
                const uint32_t at0 = __ballot_sync(0xffffffffu, first <= f0 && f0 < last);
                const uint32_t at1 = __ballot_sync(0xffffffffu, first <= f1 && f1 < last);
                const int x0 = n_first > 0 ? next_row(f0) : 0, x1 = n_first > 0 ? next_row(f1) : 0;
                f0 = at0 ? __shfl_sync(0xffffffffu, x0, __ffs(at0) - 1) : f0;
                cnt = (at1 ? __shfl_sync(0xffffffffu, x1, __ffs(at1) - 1) : total) - f0;
            } else {
                if (tid == 0) {
                    s_last[0] = f0;
                    s_last[1] = total;
                }
                __syncthreads();
                if (first <= f0 && f0 < last) s_last[0] = next_row(f0);
                if (first <= f1 && f1 < last) s_last[1] = next_row(f1);
                __syncthreads();
                f0 = s_last[0];
                cnt = s_last[1] - f0;
            }
            if (cnt <= 0) return;
        }
    }
    const int part = (cnt + W - 1) / W;
    auto claim = [&](int r, int n, int end) {                        // `end`: slices up to request r, a head
        const int lo = (end - n) * blocks - f0, hi = end * blocks - f0;
#pragma unroll 1
        for (int i = 0; i < W && n > 0; ++i)
            if (lo <= i * part && i * part < hi) {
                s_req[i] = r;
                s_off[i] = i * part - lo;
            }
    };
    int len0 = 0, r, off_r;
    if (few) {
        const int lo = (incl - n_first) * blocks - f0, hi = incl * blocks - f0, x = w * part;
        const uint32_t mine = __ballot_sync(0xffffffffu, n_first > 0 && lo <= x && x < hi && x < cnt);
        r = mine ? __ffs(mine) - 1 : -1;
        off_r = x - __shfl_sync(0xffffffffu, lo, max(r, 0));
    } else {
        claim(tid, n_first, incl);
#pragma unroll 1
        for (int base = T; base < p.requests && carry * blocks < f0 + cnt; base += T) {   // the same for all threads
            const int len = base + tid < p.requests ? attn_len(p, base + tid) : -1;
            const int n = attn_slices<TS>(p, len);
            incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            __syncthreads();                                             // s_scan and s_len have been read
            if (lane == 31) s_scan[w].x = incl;
            s_len[tid] = len;
            len0 = base;
            __syncthreads();
            int before = carry;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (i < w) before += s_scan[i].x;
                carry += s_scan[i].x;
            }
            claim(base + tid, n, before + incl);
        }
        __syncthreads();
        r = s_req[w];
        off_r = s_off[w];
    }
    auto len_of = [&](int r) { return r >= len0 && r - len0 < T ? s_len[copy + r - len0] : attn_len(p, r); };
    int left = max(0, min(part, cnt - w * part));                    // slices of this warp
    if (r < 0) left = 0;                                             // no part (or lens changed under the call)
    int h = 0, s = 0;
    if (left > 0) {
        const int ns0 = max(1, attn_slices<TS>(p, len_of(r)));
        h = off_r < ns0 ? 0 : off_r / ns0;
        s = off_r - h * ns0;
    }

    // ---- queries of a row, as they come, into q_raw ----
    auto fetch_query = [&](int row, int block) {
        const int hk = head_of(block);
        const unsigned char* src = reinterpret_cast<const unsigned char*>(
            p.q + static_cast<int64_t>(row) * p.q_stride + (static_cast<int64_t>(hk) * p.group + head0) * p.head_dim);
        const int per = p.head_dim / 4;                              // 8-byte pieces of a head
        const uint32_t to = smem_addr(q_raw);
#pragma unroll 1
        for (int hd = 0; hd < nh; ++hd)
#pragma unroll 1
            for (int i = lane; i < per; i += 32) copy8(to + hd * S::kRawStride + i * 8, src + (hd * per + i) * 8);
        if (FP8 && !BLOCK && lane < 2 && (lane ? p.v_scale : p.k_scale))
            copy4(smem_addr(&s_scales[w][lane]), (lane ? p.v_scale : p.k_scale) + hk);
        if (TMA || !kDrop) copies_arrive(smem_addr(&s_qbar[w]));
    };

    // ---- copies of K and V into this warp's ring: entries K0 V0 K1 V1 ..., E of them at a time ----
    //
    // An entry holds the rows of a slice as lines of 128 bytes (one, two or four per row, each line's rows together)
    // with 16-byte chunk c of row r at c ^ (r & 7), the tensor copies' 128-byte swizzle; rows of 64 bytes with the
    // 64-byte one. Tensor copies move boxes of slots of one page (a power of two that divides page and slice), a
    // lane per box and line. Where pages are no multiple of 8 slots, or lie outside this GPU's memory, every thread
    // copies 16-byte chunks.
    using Mask = std::conditional_t<TS == 64, uint64_t, uint32_t>;   // tokens of a slice
    constexpr Mask kAll = static_cast<Mask>(~0ull >> (64 - TS));
    constexpr int LINES = RB < 128 ? 1 : RB / 128, LB = RB < 128 ? RB : 128;
    const uint32_t ring = smem_addr(ring_p);
    const uint32_t bars = smem_addr(s_bar) + static_cast<uint32_t>(w) * E * 8;
    const int mine = left;                // slices of this warp
    const int chunks = p.head_dim * (FP8 ? 1 : 2) / 16;
    // K and V that no other CTA reads leave the L2 first where pieces of rows wait in it (wide heads in groups of 16:
    // 70.4 -> 68.0 us); elsewhere that costs up to 4% of the stream.
    const uint64_t keep = !S::kFirstShared && p.qtiles == 1 ? keep_first_out() : keep_normal();
    int issued = 0, slot_at = 0;          // slices (their K), and the next entry's place in the ring
    Mask valid_of = 0;                    // lane i: the visible tokens of slice i (modulo 32)
    int64_t off = 0;                      // of the slice whose K went out last, lane i: byte offset of token i;
    int box_page = 0, box_in = 0, box_h = 0;   // page, place in it and head of box i
    Mask last_valid = 0;                  // and its visible tokens

    // Pages are looked up for a batch of slices at a time, a lane per box (per token without tensor copies), and
    // a batch ahead: a look-up takes as long as all the copies in flight before it (3 us under load).
    const int box_shift = TMA ? p.box_shift : 0, box = 1 << box_shift;
    const int per_slice = TS >> box_shift;                           // lanes a slice
    const int slice_shift = 31 - __clz(per_slice), batch = 32 >> slice_shift;   // slices a batch
    struct Look {
        int r, h, s;                      // the slice
        int page, in;                     // in: the box's first slot in the page, -1 if no token of it is visible
        Mask valid;                       // the slice's visible tokens
    };
    Look now = {}, then = {};
    then.r = r;
    then.h = h;
    then.s = s - 1;                       // the slice before the first
    int looked = 0;                       // slices up to the end of `then`; `now` is the batch before it
    auto look_ahead = [&]() {             // `then` becomes the batch after it
        now = then;
        const int last = looked ? (batch - 1) * per_slice : 0;       // a lane of its last slice
        const int idx = lane >> slice_shift;
        int ur = __shfl_sync(0xffffffffu, then.r, last), uh = __shfl_sync(0xffffffffu, then.h, last);
        int us = __shfl_sync(0xffffffffu, then.s, last) + 1 + idx;
        then.page = then.in = -1;
        if (looked + idx < mine) {
            int len = len_of(ur), ns = max(1, attn_slices<TS>(p, len));
#pragma unroll 1
            while (us >= ns) {
                us -= ns;
                if (++uh == blocks) {
                    uh = 0;
#pragma unroll 1
                    do {
                        if (++ur >= p.requests) {                    // only if lens changed under the call
                            len = 0;
                            ns = 0x7fffffff;
                            break;
                        }
                        len = len_of(ur);
                        ns = attn_slices<TS>(p, len);
                    } while (ns == 0);
                }
            }
            const int begin = attn_begin(p, len);
            const int first = (begin / TS + us) * TS;
            const int lo = max(begin - first, 0), hi = min(len - first, TS);
            then.valid = kAll >> (TS - max(hi, 1)) & kAll << lo;     // lo < TS; hi >= 1 in a row of the list
            then.r = ur;
            then.h = uh;
            then.s = us;
            const int tok = first + ((lane & (per_slice - 1)) << box_shift);
            if (tok < len && tok + box > begin) {
                const int blk = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
                then.in = tok - blk * p.page_size;
                then.page = p.table[ur * p.table_stride + blk];
            }
        }
        looked += batch;
    };
    constexpr int LPR = CPR < 8 ? CPR : 8, RPI = 32 / LPR;
    const int crow = lane / LPR, cch = lane % LPR;
    auto copy_rows = [&](const unsigned char* base, uint32_t dst0) {
        const unsigned char* const at = base + cch * 16;
        const bool full = last_valid == kAll && chunks == CPR;
#pragma unroll
        for (int i = 0; i < TS / RPI; ++i) {
            const int row = i * RPI + crow;
            const unsigned char* const src = at + __shfl_sync(0xffffffffu, off, row);
            const int sw = CPR >= 8 ? row & 7 : (row >> 1) & 3;
            const uint32_t dst = dst0 + row * LB + ((cch ^ sw) << 4);
#pragma unroll
            for (int c = 0; c < LINES; ++c) {
                if (full) {
                    copy16(dst + c * TS * 128, src + c * 128);
                } else {
                    const bool in = (last_valid >> row & 1u) && c * LPR + cch < chunks;   // else zeros
                    copy16_or_zero(dst + c * TS * 128, in ? src + c * 128 : base, in);
                }
            }
        }
    };
    auto issue = [&](auto k_or_v) {
        constexpr bool kIsK = decltype(k_or_v)::value;
        if (issued < mine) {
            const uint32_t dst = ring + slot_at * S::kEntry, bar = bars + slot_at * 8;
            if constexpr (kIsK) {
#pragma unroll 1
                while (issued >= looked - batch) look_ahead();
                const int of = (issued & (batch - 1)) * per_slice, i = TMA ? lane / LINES : lane & (TS - 1);
                const int page = __shfl_sync(0xffffffffu, now.page, (of + i) & 31);
                const int place = __shfl_sync(0xffffffffu, now.in, (of + i) & 31);
                const int head = head_of(__shfl_sync(0xffffffffu, now.h, of));
                last_valid = __shfl_sync(0xffffffffu, now.valid, of);
                const bool has = i < per_slice && place >= 0;
                const bool in = has && page >= 0 && page < p.num_pages;
                const uint32_t bad = __ballot_sync(0xffffffffu, has && !in);
                if (bad) {                                           // their tokens count as masked
                    if (lane == 0) atomicOr(&g_attn_status, kStatusBadPage);
                    const int lines = TMA ? LINES : 1;
#pragma unroll 1
                    for (int k = 0; k < TS; ++k)
                        if (bad >> ((k >> box_shift) * lines) & 1u) last_valid &= ~(Mask(1) << k);
                }
                if (lane == (issued & 31)) valid_of = last_valid;
                if constexpr (BLOCK) {                               // the scales of tokens lane, lane + 32
                    const uint32_t to = smem_addr(smem + S::kScalesAt + w * S::kScales +
                                                  (issued & (S::kScalePlaces - 1)) * TS * 8);
#pragma unroll
                    for (int x = 0; x < (TS + 31) / 32; ++x) {
                        const int tok = x * 32 + lane, b = of + (tok >> box_shift);
                        const int64_t pg = __shfl_sync(0xffffffffu, now.page, b & 31);
                        const int slot = __shfl_sync(0xffffffffu, now.in, b & 31) + (tok & (box - 1));
                        const bool seen = tok < TS && (last_valid >> (tok & (TS - 1)) & 1u);
                        const int blk = p.block_shift >= 0 ? slot >> p.block_shift : slot / p.block_tokens;
                        const int64_t at = seen ? pg * p.scale_page_stride + blk * p.scale_block_stride +
                                                      head * p.scale_head_stride : 0;
                        if (tok < TS) {
                            copy4_or_zero(to + tok * 8, p.k_block_scale + at, seen);
                            copy4_or_zero(to + tok * 8 + 4, p.v_block_scale + at, seen);
                        }
                    }
                    if constexpr (TMA) copies_arrive(bar);
                }
                if constexpr (TMA) {
                    box_page = in ? page : p.num_pages;              // outside the view: zeros
                    box_in = in ? place : 0;
                    box_h = head;
                } else {
                    off = in ? page * p.page_stride + head * p.head_stride + place * p.slot_stride : 0;
                }
            }
            if constexpr (TMA) {
                // Boxes without a visible token are left out with a scale for each block: their scores are masked, their
                // rows of V zeroed below, and copying zeros took as long as a box does (179 x 22 tokens in pages of 24
                // slots 16.4 -> 9.8 us).
                const bool in_slice = lane < per_slice * LINES && (!BLOCK || box_page < p.num_pages);
                const uint32_t boxes = __ballot_sync(0xffffffffu, in_slice);
                if (lane == 0) expect_bytes(bar, BLOCK ? __popc(boxes) * LB << box_shift : S::kEntry);
                __syncwarp();
                if (in_slice && (kIsK || !kDrop))
                    copy_box(dst + lane % LINES * TS * 128 + lane / LINES * box * LB, kIsK ? &p.kmap : &p.vmap,
                             lane % LINES * (FP8 ? 128 : 64), box_in, box_h, box_page, bar, keep);
            } else {
                copy_rows(kIsK ? p.kc : p.vc, dst);
                copies_arrive(bar);
            }
        }
        if constexpr (!kIsK) ++issued;
        slot_at = slot_at + 1 == E ? 0 : slot_at + 1;
    };
    using K = std::true_type;
    using V = std::false_type;
    if (mine > 0) {
        look_ahead();                     // the first pages are on their way,
        fetch_query(attn_row(p, r), h);   // and the first row's queries
    }
#pragma unroll 1
    for (int i = 0; i < E; ++i) {
        if (i & 1) issue(V{});
        else issue(K{});
    }
    int taken = 0, take_at = 0;           // slices; the next entry's place in the ring, and its barrier's phase
    uint32_t phase = 0;
    bool ok = true;
    auto landed = [&](bool before) {      // the next entry, for all lanes alike
        return __all_sync(0xffffffffu, before && wait_phase(bars + take_at * 8, phase)) != 0;
    };
    auto next_entry = [&]() {
        if (++take_at == E) {
            take_at = 0;
            phase ^= 1u;
        }
    };

    // ---- query fragments (B operand: 16 columns of the head x 8 heads) as the products take them ----
    constexpr int QN = S::kQueryShared ? 1 : NB;
    uint32_t qf[QN][KS][2];
    float col_scale[NB][2];
    uint32_t q_phase = 0;
    // Scores leave the first product as powers of two, or (capped) as the argument of tanh.
    const float score_scale = p.softcap > 0.f ? p.scale / p.softcap : p.scale * kLog2e;
    const float cap_log2 = p.softcap * kLog2e;
    auto raw_query = [&](int ks, int nb) {
        const unsigned char* at = q_raw + (nb * 8 + g) * S::kRawStride + ks * 32;
        if constexpr (FP8) return *reinterpret_cast<const uint2*>(at + 8 * t);
        else return make_uint2(*reinterpret_cast<const uint32_t*>(at + 4 * t),
                               *reinterpret_cast<const uint32_t*>(at + 16 + 4 * t));
    };
    float v_scale = BLOCK ? 0x1p20f : 1.f;
    auto place_query = [&]() {
        ok = __all_sync(0xffffffffu, ok && wait_phase(smem_addr(&s_qbar[w]), q_phase)) != 0;
        q_phase ^= 1u;
        const float ksc = score_scale * (FP8 ? s_scales[w][0] : 1.f);
        if constexpr (FP8 && !BLOCK) v_scale = s_scales[w][1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            col_scale[nb][0] = col_scale[nb][1] = ksc;
            uint32_t f[KS][2];
            if constexpr (!S::kQueryShared || FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint2 v = raw_query(ks, nb);
                    f[ks][0] = v.x;
                    f[ks][1] = v.y;
                }
            }
            if constexpr (FP8) {
                // The FP8 cache is widened to FP16 (exact); q is brought to FP16 by a power of two per head
                // that puts its largest value in [2^14, 2^15): what that loses is below 2^-38 of that value.
                float top = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        top = fmaxf(top, fmaxf(fabsf(low_bf16(f[ks][b])), fabsf(high_bf16(f[ks][b]))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
                e = (top > 0.f ? max(-112, min(127, e)) : 0) - 14;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        f[ks][b] = pack_f16(low_bf16(f[ks][b]) * down, high_bf16(f[ks][b]) * down);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                for (int j = 0; j < 2; ++j) col_scale[nb][j] *= __shfl_sync(0xffffffffu, up, 8 * t + 4 * j);
                if constexpr (S::kQueryShared) {                     // in place: each lane what it read
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        *reinterpret_cast<uint2*>(q_raw + (nb * 8 + g) * S::kRawStride + ks * 32 + 8 * t) =
                            make_uint2(f[ks][0], f[ks][1]);
                }
            }
            if constexpr (!S::kQueryShared) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qf[nb][ks][0] = f[ks][0];
                    qf[nb][ks][1] = f[ks][1];
                }
            }
        }
        __syncwarp();                                                // q_raw has been read
    };
    auto query = [&](int ks, int nb) {
        if constexpr (S::kQueryShared) return raw_query(ks, nb);
        else return make_uint2(qf[nb][ks][0], qf[nb][ks][1]);
    };

    auto first_piece = [&](int warp) {
        if constexpr (S::kFirstShared) return reinterpret_cast<float*>(smem + S::kRing + W * S::kRaw + warp * S::kFirst);
        else return p.part_warp + (static_cast<int64_t>(blockIdx.x) * W + warp) * H * DT;
    };

    // ---- the rows of this warp's part, one after the other ----
    int at = w * part;
    while (left > 0) {
        const int len = len_of(r);
        const int ns = attn_slices<TS>(p, len);
        const int seg = min(ns - s, left);
        if (seg <= 0) break;                                         // only if lens changed under the call
        const int row = attn_row(p, r);
        place_query();

        // The row after this one.
        int next_r = r, next_h = h;
        if (seg < left && ++next_h == blocks) {
            next_h = 0;
#pragma unroll 1
            do ++next_r;
            while (next_r < p.requests && attn_slices<TS>(p, len_of(next_r)) == 0);
        }
        const bool more = seg < left && next_r < p.requests;
        if (!S::kQueryShared && more) fetch_query(attn_row(p, next_r), next_h);

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

#pragma unroll 1
        for (int step = 0; step < seg; ++step) {
            if (!(ok = landed(ok))) break;
            const Mask valid = __shfl_sync(0xffffffffu, valid_of, taken & 31);

            // S^T = K Q^T: rows g and g + 8 of a tile are tokens, columns 2t and 2t + 1 heads.
            float sc[MT][NB][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) sc[mt][nb][0] = sc[mt][nb][1] = sc[mt][nb][2] = sc[mt][nb][3] = 0.f;
            {
                const uint32_t kb = ring + take_at * S::kEntry;
                const int arow = lane & 15;
                const int asw = CPR >= 8 ? arow & 7 : (arow >> 1) & 3;
#pragma unroll
                for (int c = 0; c < CPR; c += 2) {                   // two 16-byte chunks of the rows
                    uint32_t a[MT][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        ldsm4(a[mt], kb + c / 8 * TS * 128 + (mt * 16 + arow) * LB +
                                         (((c % 8 + (lane >> 4)) ^ asw) << 4));
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
                                e4m3_to_f16(a[mt][2 * x], f[mt][0], f[mt][2]);
                                e4m3_to_f16(a[mt][2 * x + 1], f[mt][1], f[mt][3]);
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
            // Scales of the tokens of this lane's rows: of k, the logarithm of that of v, and that of v itself by what the
            // sum is kept larger.
            float ks[BLOCK ? MT : 1][2], lv[BLOCK ? MT : 1][2], vs[BLOCK ? MT : 1][2];
            if constexpr (BLOCK) {
                const float2* const at = reinterpret_cast<const float2*>(smem + S::kScalesAt + w * S::kScales) +
                                         (taken & (S::kScalePlaces - 1)) * TS;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 of = at[mt * 16 + j * 8 + g];
                        const float v_of = of.y < 0x1p-60f ? 0x1p-60f : of.y;
                        ks[mt][j] = fmaf(of.y, 0.f, of.x);           // NaN where that of v is NaN, so that the sum is too
                        lv[mt][j] = log2_ftz(v_of);
                        vs[mt][j] = v_of * 0x1p-20f;
                    }
            }
            __syncwarp();
            next_entry();
            issue(std::bool_constant<E % 2 == 0>{});                 // into the entry just read: E entries on

            // Running maximum and sum, in powers of two.
            uint32_t pb[MT][NB][2], pl[FP8 ? 1 : MT][FP8 ? 1 : NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float x[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[mt][j] = sc[mt][nb][j] * col_scale[nb][j & 1];
                        if constexpr (BLOCK) x[mt][j] *= ks[mt][j >> 1];
                    }
                if (p.softcap > 0.f) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[mt][j] = cap_log2 * tanhf(x[mt][j]);
                }
                if (valid != kAll) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (!(valid >> (mt * 16 + g + (j & 2) * 4) & 1u)) x[mt][j] = kNegInf;
                }
                float corr[2], base[2], shift[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    auto term = [&](int mt, int i) {
                        if constexpr (BLOCK) return x[mt][i] + lv[mt][i >> 1];
                        else return x[mt][i];
                    };
                    float top = fmaxf(term(0, j), term(0, j + 2));
                    #pragma unroll
                    for (int mt = 1; mt < MT; ++mt) top = fmaxf(top, fmaxf(term(mt, j), term(mt, j + 2)));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[nb][j]);
                    base[j] = base_of(top);
                    shift[j] = top == INFINITY ? 0.f : m[nb][j] - base[j];            // this lane's l may be 0
                    corr[j] = exp2_ftz(shift[j]);
                    m[nb][j] = top;
                }
                if constexpr (!BLOCK) {
                    l[nb][0] *= corr[0];
                    l[nb][1] *= corr[1];
                }
                if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        acc[ks][nb][0] *= corr[0];
                        acc[ks][nb][1] *= corr[1];
                        acc[ks][nb][2] *= corr[0];
                        acc[ks][nb][3] *= corr[1];
                    }
                    if constexpr (BLOCK) {
                        l[nb][0] = moved(l[nb][0], shift[0], corr[0]);
                        l[nb][1] = moved(l[nb][1], shift[1], corr[1]);
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[mt][j] = exp2_ftz(x[mt][j] - (base[j & 1] - kSumUp));
                    l[nb][0] += x[mt][0] + x[mt][2];
                    l[nb][1] += x[mt][1] + x[mt][3];
                    if constexpr (BLOCK) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[mt][j] *= vs[mt][j >> 1];
                    }
                    // P as the B operand. FP16 beside an FP8 cache (2^-11 relative, down to 2^-29 of the largest
                    // weight). Beside a BF16 cache P has to be BF16, whose 2^-8 would double the rounding error of
                    // a BF16 output: it goes in two parts, the BF16 number below it and the rest in a second one,
                    // 2^-16 together. Both are above zero (down to 2^-110 of the largest weight, where the rest
                    // leaves BF16's range), so that an infinite v stays what it is: 0 * inf and inf - inf are NaN.
                    if constexpr (FP8) {
                        pb[mt][nb][0] = transpose8x8(pack_f16(x[mt][0], x[mt][1]));
                        pb[mt][nb][1] = transpose8x8(pack_f16(x[mt][2], x[mt][3]));
                    } else {
                        constexpr float kBelow = 1.f - 0x1p-23f;                  // to the next FP32 number or two below
                        const uint32_t a = pack_bf16_down(x[mt][0] * kBelow, x[mt][1] * kBelow);
                        const uint32_t b = pack_bf16_down(x[mt][2] * kBelow, x[mt][3] * kBelow);
                        pb[mt][nb][0] = transpose8x8(a);
                        pb[mt][nb][1] = transpose8x8(b);
                        pl[mt][nb][0] = transpose8x8(pack_bf16(x[mt][0] - low_bf16(a), x[mt][1] - high_bf16(a)));
                        pl[mt][nb][1] = transpose8x8(pack_bf16(x[mt][2] - low_bf16(b), x[mt][3] - high_bf16(b)));
                    }
                }
            }

            // O^T += V^T P^T: rows are columns of the head.
            if (!(ok = landed(ok))) break;
            const uint32_t vb = ring + take_at * S::kEntry;
            if (TMA && valid != kAll) {
                // A box brings whole rows of the page, also those past the length: 0 * NaN must not get into the sum.
#pragma unroll 1
                for (int row = lane; row < TS; row += 32)
                    if (!(valid >> row & 1u)) {
#pragma unroll 1
                        for (int c = 0; c < CPR; ++c) {
                            const uint32_t to = vb + c / 8 * TS * 128 + row * LB + (c % 8) * 16;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(to), "r"(0) : "memory");
                        }
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the entry's next copy
                __syncwarp();
            }
            if constexpr (!FP8) {
                const int vrow = (lane & 7) + ((lane >> 4) << 3);
                const int vsw = vrow & 7;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        ldsm4_t(a, vb + ks / 4 * TS * 128 + (mt * 16 + vrow) * LB +
                                       (((2 * ks % 8 + ((lane >> 3) & 1)) ^ vsw) << 4));
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
                        ldsm4_t(a, vb + c / 8 * TS * 128 + (mt * 16 + vrow) * LB +
                                       (((c % 8 + (lane >> 4)) ^ vsw) << 4));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_f16(__byte_perm(a[2 * x], 0, 0x3120), a0, a1);
                            e4m3_to_f16(__byte_perm(a[2 * x + 1], 0, 0x3120), a2, a3);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma<true>(acc[c + x][nb], a0, a1, a2, a3, pb[mt][nb][0], pb[mt][nb][1]);
                        }
                    }
            }
            __syncwarp();
            ++taken;
            next_entry();
            issue(std::bool_constant<E % 2 == 1>{});
        }
        if (!ok) {                                                   // a copy never came: no plausible numbers
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                m[nb][0] = m[nb][1] = 0.f;
                l[nb][0] = l[nb][1] = __int_as_float(0x7fffffff);
            }
        }
        if (S::kQueryShared && more) fetch_query(attn_row(p, next_r), next_h);

        // ---- what becomes of the row ----
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 4);
                l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 8);
                l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 16);
            }
        const bool whole = s == 0 && seg == ns, final = seg == left;
        if (whole) {
            const int64_t head_at = static_cast<int64_t>(head_of(h)) * p.group + head0;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float inv[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int hd = nb * 8 + 2 * t + j;
                    inv[j] = l[nb][j] == 0.f ? 0.f : v_scale / l[nb][j];
                    if (l[nb][j] == 0.f) {                           // no weight at all: zeros, whatever v holds
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) acc[ks][nb][j] = acc[ks][nb][j + 2] = 0.f;
                    }
                    // No weight: -inf. NaN scores, which no maximum shows, have made the sum NaN.
                    if (p.lse && g == 0 && hd < nh)
                        p.lse[static_cast<int64_t>(row) * p.q_heads + head_at + hd] =
                            (m[nb][j] + log2f(l[nb][j] * kSumDown)) * kLn2;
                }
                // Transposed again, lane (g, t) holds columns 2t, 2t + 1 of the tile's rows for head g.
                uint16_t* const o = p.out + static_cast<int64_t>(row) * p.out_stride + (head_at + nb * 8 + g) * p.head_dim;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t a = transpose8x8(pack_bf16(acc[ks][nb][0] * inv[0], acc[ks][nb][1] * inv[1]));
                    const uint32_t b = transpose8x8(pack_bf16(acc[ks][nb][2] * inv[0], acc[ks][nb][3] * inv[1]));
                    if (nb * 8 + g < nh && ks * 16 < p.head_dim) {
                        if constexpr (FP8) {                         // a: even columns, b: odd ones
                            *reinterpret_cast<uint2*>(o + ks * 16 + 4 * t) =
                                make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
                        } else {
                            *reinterpret_cast<uint32_t*>(o + ks * 16 + 2 * t) = a;
                            if (ks * 16 + 8 < p.head_dim) *reinterpret_cast<uint32_t*>(o + ks * 16 + 8 + 2 * t) = b;
                        }
                    }
                }
            }
        } else {
            // A piece: the last one to the warp's ring, whose copies are all consumed.
            float* const o = final ? reinterpret_cast<float*>(ring_p) : first_piece(w);
            float2* const ml = s_ml[2 * w + (final ? 1 : 0)];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int hd = nb * 8 + 2 * t + j;
                    if (hd < nh) {
                        if (g == 0) ml[hd] = make_float2(m[nb][j], l[nb][j]);
                        // Column d of head hd at d ^ 8 t: the four heads a store covers lie in different banks.
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            const int d0 = ks * 16 + (FP8 ? 2 * g : g), d1 = FP8 ? d0 + 1 : d0 + 8;
                            o[hd * DT + (d0 ^ 8 * t)] = acc[ks][nb][j];
                            o[hd * DT + (d1 ^ 8 * t)] = acc[ks][nb][j + 2];
                        }
                    }
                }
            if (lane == 0) s_piece[2 * w + (final ? 1 : 0)] = {1, r, h, s, seg, ns, at, row, v_scale};
        }

        left -= seg;
        at += seg;
        s = 0;                                                       // a part that goes on, goes on with a new row
        r = next_r;
        h = next_h;
        if (!more) break;
    }
    // After a timed-out wait: give this warp's other copies in flight the same time to land.
    if (!ok)
        for (int i = 0; i < E && wait_phase(bars + take_at * 8, phase); ++i) next_entry();
    __syncthreads();

    // ---- the warps' pieces, joined row by row ----
    auto store = [&](int row, int block, int hd, int d, float4 o, float top, float sum, float scale) {
        const int64_t head = static_cast<int64_t>(head_of(block)) * p.group + head0 + hd;
        const float inv = sum == 0.f ? 0.f : scale / sum;
        if (sum == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(row) * p.out_stride + head * p.head_dim + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (p.lse && d == 0)
            p.lse[static_cast<int64_t>(row) * p.q_heads + head] = (top + log2f(sum * kSumDown)) * kLn2;
    };
    const int d4s = p.head_dim / 4, items = nh * d4s;
    auto head_at = [&](int x) { return static_cast<int>(x * p.quarter_of >> 20); };   // x / d4s
    // Every warp finds the rows among the pieces by itself: lane i holds piece i.
    Piece own = {0, -1, -1, 0, 0, 0, 0, 0, 1.f};
    if (lane < 2 * W) own = s_piece[lane];
    const uint32_t pieces = __ballot_sync(0xffffffffu, own.valid != 0);
    uint32_t starts;                      // the first piece of each row
    {
        const uint32_t before = pieces & ((1u << lane) - 1u);
        const int prev = before ? 31 - __clz(before) : 0;
        const int pr = __shfl_sync(0xffffffffu, own.r, prev), ph = __shfl_sync(0xffffffffu, own.h, prev);
        starts = __ballot_sync(0xffffffffu, own.valid != 0 && (!before || pr != own.r || ph != own.h));
    }
    auto piece_at = [&](int i) {
        Piece a;
        a.valid = 1;
        a.r = __shfl_sync(0xffffffffu, own.r, i);
        a.h = __shfl_sync(0xffffffffu, own.h, i);
        a.s = __shfl_sync(0xffffffffu, own.s, i);
        a.seg = __shfl_sync(0xffffffffu, own.seg, i);
        a.ns = __shfl_sync(0xffffffffu, own.ns, i);
        a.at = __shfl_sync(0xffffffffu, own.at, i);
        a.row = __shfl_sync(0xffffffffu, own.row, i);
        a.v_scale = __shfl_sync(0xffffffffu, own.v_scale, i);
        return a;
    };
    Piece before = {}, after = {};        // the rows that go on in other CTAs: one from before, one after
    constexpr int UW = (H * DT / 4 + T - 1) / T;                     // units of 32 items that a warp takes of a row
#pragma unroll 1
    for (uint32_t rest = starts; rest;) {
        const int i = __ffs(rest) - 1;
        rest &= rest - 1;
        const uint32_t of = pieces & (0xffffffffu << i) & (rest ? (1u << (__ffs(rest) - 1)) - 1u : 0xffffffffu);
        // The row's pieces: i, i + 2, .. the last ones of consecutive warps, and j, the last or the first of the
        // warp where the row (or the range) ends.
        const int j = 31 - __clz(of), n = __popc(of);
        const Piece a = piece_at(i);
        const int reach = __shfl_sync(0xffffffffu, own.s + own.seg, j);
        const bool whole = a.s == 0 && reach == a.ns;
        if (!whole) (a.s == 0 ? after : before) = a;
        const int64_t piece = static_cast<int64_t>(blockIdx.x) * 2 + (a.s == 0 ? 1 : 0);
        // Piece j first: it may have to come from the workspace, all of this warp's share at once.
        float4 tail[UW];
#pragma unroll
        for (int u = 0; u < UW; ++u) {
            const int x = u * T + tid, hd = head_at(x), d = (x - hd * d4s) * 4;
            const float* from = j & 1 ? reinterpret_cast<const float*>(smem + (j >> 1) * kAttnRing) : first_piece(j >> 1);
            if (x < items) tail[u] = *reinterpret_cast<const float4*>(from + hd * DT + (d ^ (hd >> 1 & 3) * 8));
        }
#pragma unroll
        for (int u = 0; u < UW; ++u) {
            const int x = u * T + tid;
            if (x >= items) break;
            const int hd = head_at(x), d = (x - hd * d4s) * 4;
            const int place = hd * DT + (d ^ (hd >> 1 & 3) * 8);
            const float2 ml_j = s_ml[j][hd];
            float2 ml[W - 1];
            float top = ml_j.x;
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                ml[k] = k < n - 1 ? s_ml[i + 2 * k][hd] : make_float2(kNegInf, 0.f);
                top = fmaxf(top, ml[k].x);
            }
            const float base = base_of(top);
            float e = exp2_ftz(ml_j.x - base);
            float sum = moved(ml_j.y, ml_j.x - base, e);
            float4 o = make_float4(tail[u].x * e, tail[u].y * e, tail[u].z * e, tail[u].w * e);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                if (k < n - 1) {
                    const float4 v = *reinterpret_cast<const float4*>(smem + ((i >> 1) + k) * kAttnRing + place * 4);
                    e = exp2_ftz(ml[k].x - base);
                    sum += moved(ml[k].y, ml[k].x - base, e);
                    o.x += v.x * e;
                    o.y += v.y * e;
                    o.z += v.z * e;
                    o.w += v.w * e;
                }
            if (whole) {
                store(a.row, a.h, hd, d, o, top, sum, a.v_scale);
            } else {
                *reinterpret_cast<float4*>(p.part + (piece * H + hd) * DT + d) = o;
                if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (piece * H + hd) * 2) = make_float2(top, sum);
            }
        }
    }
    if (!before.valid && !after.valid) return;

    // ---- rows cut between CTAs: the CTA that arrives last joins their pieces ----
    //
    // A row of more than kJoin pieces is joined in groups first, each by the last of its CTAs to arrive, and the
    // groups' results by the last group. Piece 1 of a row's first CTA, piece 0 of the others; a group's result takes
    // the place of its last piece.
    constexpr int kJoin = 32;
    __syncthreads();                      // the CTA's pieces are written; whoever counts it in makes them visible
    // The first and last CTA of the row from before (lanes 0 and 1), of the one after (lanes 2 and 3).
    const Piece cut = lane < 2 ? before : after;
    const int row0 = f0 + cut.at - cut.s;                            // where it starts in the list
    int ends = first_of_row + (lane & 1 ? per_row - 1 : 0);
    if (per_row == 0) ends = (row0 + (lane & 1 ? cut.ns - 1 : 0)) / quota;
    const int from0 = __shfl_sync(0xffffffffu, ends, 0), to0 = __shfl_sync(0xffffffffu, ends, 1);
    const int from1 = __shfl_sync(0xffffffffu, ends, 2), to1 = __shfl_sync(0xffffffffu, ends, 3);
    // One more arrival at a counter; whether it is the last of `all`, with the counter zero again for the next call.
    // By one thread behind a barrier of the CTA, before and after: its fences stand for all threads.
    auto arrive = [&](uint32_t* ticket, int all) {
        __threadfence();
        const bool last = atomicAdd(ticket, 1u) == static_cast<uint32_t>(all - 1);
        if (last) {
            *ticket = 0u;
            __threadfence();
        }
        return last;
    };
    enum { kWait, kLast, kGroups };
    if (lane == 0 && w < 2) {
        int state = kWait;
        if (w == 0 ? before.valid : after.valid) {
            const int from = w == 0 ? from0 : from1, n = (w == 0 ? to0 : to1) - from + 1;
            state = n > kJoin ? kGroups : arrive(p.ticket + place_of(from), n) ? kLast : kWait;
        }
        s_last[w] = state;
    }
    __syncthreads();

    // Joins the pieces of CTAs c0, c0 + 2^step_shift, .. up to `end` (the last one always `end`). Narrow tiles leave
    // threads over: `parts` threads share an item then, each with every parts-th piece (from mine_of, past them:
    // idle), and meet in the ring. B at a time, all of whose loads are in flight together.
    constexpr int B = UW == 1 ? 5 : UW == 2 ? 8 : 4;
    const int parts = UW > 1 || 2 * items > T ? 1 : 4 * items > T ? 2 : 4;
    const int mine_of = UW > 1 ? 0 : (tid >= items) + (tid >= 2 * items) + (tid >= 3 * items) + (tid >= 4 * items);
    const int item = tid - mine_of * items;
    float top[UW], sum[UW];
    float4 o[UW];
    auto join = [&](int from, int c0, int step_shift, int end) {
        const int count = ((end - c0 + (1 << step_shift) - 1) >> step_shift) + 1;
#pragma unroll
        for (int u = 0; u < UW; ++u) {
            top[u] = kNegInf;
            sum[u] = 0.f;
            o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int b0 = mine_of; b0 < count && mine_of < parts; b0 += B * parts) {
            float2 ml[B][UW];
            float4 v[B][UW];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int at_b = b0 + b * parts, c = min(c0 + (at_b << step_shift), end);
                const int at = (place_of(c) * 2 + (c == from ? 1 : 0)) * H;   // heads of pieces: below 2^31
#pragma unroll
                for (int u = 0; u < UW; ++u) {
                    const int x = u * T + item, hd = head_at(x), d = (x - hd * d4s) * 4;
                    ml[b][u] = make_float2(kNegInf, 0.f);
                    v[b][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (at_b < count && x < items) {
                        ml[b][u] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at + hd);
                        v[b][u] = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(at + hd) * DT + d));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < UW; ++u) {
                float next = top[u];
#pragma unroll
                for (int b = 0; b < B; ++b) next = fmaxf(next, ml[b][u].x);
                const float base = base_of(next), e = exp2_ftz(top[u] - base);
                sum[u] = moved(sum[u], top[u] - base, e);
                o[u] = make_float4(o[u].x * e, o[u].y * e, o[u].z * e, o[u].w * e);
                top[u] = next;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const float f = exp2_ftz(ml[b][u].x - base);
                    sum[u] += moved(ml[b][u].y, ml[b][u].x - base, f);
                    o[u].x += v[b][u].x * f;
                    o[u].y += v[b][u].y * f;
                    o[u].z += v[b][u].z * f;
                    o[u].w += v[b][u].w * f;
                }
            }
        }
        if constexpr (UW == 1) {
            if (parts == 1) return;
            float4* const s_o = reinterpret_cast<float4*>(smem);
            float2* const s_x = reinterpret_cast<float2*>(smem + T * 16);
            __syncthreads();                                         // the ring has been read
            s_o[tid] = o[0];
            s_x[tid] = make_float2(top[0], sum[0]);
            __syncthreads();
            if (mine_of != 0) return;
#pragma unroll 1
            for (int k = 1; k < parts; ++k) {
                const float2 ml = s_x[k * items + tid];
                const float4 v = s_o[k * items + tid];
                const float next = fmaxf(top[0], ml.x), base = base_of(next);
                const float e = exp2_ftz(top[0] - base), f = exp2_ftz(ml.x - base);
                sum[0] = moved(sum[0], top[0] - base, e) + moved(ml.y, ml.x - base, f);
                top[0] = next;
                o[0].x = o[0].x * e + v.x * f;
                o[0].y = o[0].y * e + v.y * f;
                o[0].z = o[0].z * e + v.z * f;
                o[0].w = o[0].w * e + v.w * f;
            }
        }
    };
    auto store_row = [&](const Piece& a) {
#pragma unroll
        for (int u = 0; u < UW; ++u) {
            const int x = u * T + tid, hd = head_at(x);
            if (x < items) store(a.row, a.h, hd, (x - hd * d4s) * 4, o[u], top[u], sum[u], a.v_scale);
        }
    };
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (s_last[k] != kLast) continue;
        const int from = k == 0 ? from0 : from1, to = k == 0 ? to0 : to1;
        join(from, from, 0, to);
        store_row(k == 0 ? before : after);
    }
    if (s_last[0] != kGroups && s_last[1] != kGroups) return;
    const bool big[2] = {s_last[0] == kGroups, s_last[1] == kGroups};
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? big[0] : big[1])) continue;
        const int from = k == 0 ? from0 : from1, to = k == 0 ? to0 : to1, n = to - from + 1;
        const int gs = n <= 64 ? 3 : n <= 256 ? 4 : 5, groups = (n + (1 << gs) - 1) >> gs;
        const int begin = from + ((cta - from) >> gs << gs), end = min(begin + (1 << gs) - 1, to);
        // Groups are counted at their last CTA, which no other row's group ends at.
        __syncthreads();                                             // s_last has been read
        if (tid == 0) s_last[k] = arrive(p.ticket + kAttnTickets / 2 + place_of(end), end - begin + 1);
        __syncthreads();
        if (!s_last[k]) continue;
        join(from, begin, 0, end);
        __syncthreads();                                             // every thread has read the group's pieces
#pragma unroll
        for (int u = 0; u < UW; ++u) {
            const int x = u * T + tid, hd = head_at(x), d = (x - hd * d4s) * 4;
            if (x >= items) break;
            const int64_t at = static_cast<int64_t>(place_of(end)) * 2 * H + hd;
            *reinterpret_cast<float4*>(p.part + at * DT + d) = o[u];
            if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(top[u], sum[u]);
        }
        __syncthreads();
        if (tid == 0) s_last[k] = arrive(p.ticket + place_of(from), groups);
        __syncthreads();
        if (!s_last[k]) continue;
        join(-1, from + (1 << gs) - 1, gs, to);
        store_row(k == 0 ? before : after);
    }
}

}  // namespace gemv
