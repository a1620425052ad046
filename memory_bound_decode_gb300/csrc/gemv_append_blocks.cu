// Rotary positions and the write into an FP8 cache with a scale for each block
// of tokens and head.
//
//   a = max |x| over the finite values of the new rows of a block and head,
//   need = max(2^-30, the smallest power of two >= a / 448),
//   scale' = need where the rows begin the block, else max(need, scale rounded up to a power of two),
//   code = e4m3(x / scale'); earlier codes of the block: e4m3(code * scale / scale').
//
// Scales are powers of two: dividing by one is exact, and so is moving codes to
// a larger one, but for those that fall among the subnormals.
//
// A block's scale belongs to all its tokens, so its new rows (a run of
// neighbours in the batch) have one owner, the CTA whose window of tokens the
// run begins in; the slots alone tell where that is (the block's first slot, or
// a slot that does not follow the token's before it). A few CTAs share the runs
// and heads of a window; those for which it has no work end at once. A team of
// warps takes a run and a head, as many as keep its rows in shared memory (four
// groups of 32 bytes a lane) while they look for the largest value: rows are read
// once, and what is in flight takes no registers. Single tokens (a decode step)
// take the lanes that hold a row, and registers.
//
// Measured: 4,051 tokens (4,084 rows) of 32 + 8 + 8 FP32 heads of 128 in blocks of
// 16 (141 MB) 25.7 us, 5.5 TB/s, of which 2 are the launch (issue 59% busy; BF16
// rows 18.5); 1,021 BF16 tokens in blocks of 64 9.7 us. Single tokens, in a
// replayed graph: 16 2.5 us, 254 4.8 us where no scale grows (launch, then slots
// and rows one after the other), 5.3 and 12.2 us where a quarter of the blocks
// do, 5.6 and 15.2 us where all do (then the codes of their earlier tokens).
#include <algorithm>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"
#include "gemv_common.cuh"
#include "gemv_rows.cuh"

namespace gemv {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kQueryTokens = 2;        // tokens whose query rows a thread has in flight, in registers
constexpr int kStreamTokens = 4;       // and in shared memory
// CTAs of an SM, which say how many registers a thread has, where a CTA of queries takes `tokens` of them: four where rows
// stream (three: 4,000 FP32 tokens 25.5 -> 26.3 us, BF16 17.7 -> 18.8) and for 1,021 FP32 ones (8.4 -> 8.9, but 500 6.3 -> 5.6),
// else three (four: single tokens of 254 requests 4.7 -> 5.4, 1,021 BF16 tokens 7.9 -> 8.8, in blocks of 64 9.8 -> 10.9).
constexpr int append_ctas(bool f32, int tokens) {
    return tokens == kStreamTokens || (f32 && tokens == kQueryTokens) ? 4 : 3;
}
constexpr int kMaxWindow = 32;         // tokens of a CTA that writes blocks
constexpr int kMostShared = 8 * 8192 + (kMaxWindow - 1 + GEMV_MAX_BLOCK_TOKENS) * GEMV_MAX_HEAD_DIM / 2 * 8;   // bytes
static_assert(kMaxWindow + GEMV_MAX_BLOCK_TOKENS <= 96 && kMaxWindow <= 32, "three ballots cover the tokens of a window");

// How a launch is laid out: the first kv_ctas CTAs write blocks, the others turn queries.
struct AppendShape {
    unsigned kv_ctas;
    int window;                        // tokens of a CTA that writes blocks
    int kv_parts, kv_shift;            // CTAs that share a window's heads: the first half k's, the others v's
    int groups, across;                // of a head; tokens that a warp takes side by side
    int tokens_held;                   // of a head, by a warp
    uint32_t per_group, per_head;      // u * per_group >> 32 is u / groups (groups > 1), with per_head u / kv_heads
    int turns, shared;                 // cosines in shared memory; its bytes
    int parts, parts_shift, visit;     // CTAs of a token's queries, query heads of each
};

// Cosine and sine of a position times a frequency, as in gemv_rope: the angle as a 64-bit fraction of a turn, reduced
// exactly.
__device__ __forceinline__ float2 turn_of(int32_t pos, uint64_t freq) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * freq;
    float2 cs;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &cs.y, &cs.x);
    return cs;
}

// The pairs of a group turned: x and y hold their first and second columns, or (interleaved) 2 * VEC neighbouring ones.
template <int VEC>
__device__ __forceinline__ void turn_group(float (&x)[VEC], float (&y)[VEC], bool interleaved, const float (&cs)[VEC],
                                           const float (&sn)[VEC]) {
    if (VEC == 1 || !interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float u = x[j], v = y[j];
            x[j] = u * cs[j] - v * sn[j];
            y[j] = v * cs[j] + u * sn[j];
        }
    } else if constexpr (VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {                              // the first half of the pairs in x, the others in y
            float& e = j < VEC / 2 ? x[2 * j] : y[2 * j - VEC];
            float& f = j < VEC / 2 ? x[2 * j + 1] : y[2 * j + 1 - VEC];
            const float u = e, v = f;
            e = u * cs[j] - v * sn[j];
            f = v * cs[j] + u * sn[j];
        }
    }
}

// N neighbouring values from shared memory, 16 bytes at a time (where N is 1: alone).
template <int N>
__device__ __forceinline__ void load_floats(const float* at, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = *at;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(at)[i];
            f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
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
__device__ __forceinline__ uint4 move_codes(uint4 v, float by) {
    return make_uint4(move_codes(v.x, by), move_codes(v.y, by), move_codes(v.z, by), move_codes(v.w, by));
}

// The codes of `tokens` slots from `at` on times `by`, this thread's share of them: 16 bytes each, kMoved at a time in flight
// (one after the other: a decode step of 254 tokens 8.8 us, so 5.9).
constexpr int kMoved = 4;
__device__ __noinline__ void move_block(unsigned char* at, int64_t slot_stride, int tokens, int head_dim, float by,
                                           int thread, int threads) {
    const int per = head_dim / 16, all = tokens * per;
    for (int base = thread; base < all; base += kMoved * threads) {
        uint4 w[kMoved];
        uint4* to[kMoved];
#pragma unroll
        for (int i = 0; i < kMoved; ++i) {
            const int v = min(base + i * threads, all - 1), tk = v / per;
            to[i] = reinterpret_cast<uint4*>(at + tk * slot_stride + (v - tk * per) * 16);
            w[i] = *to[i];
        }
#pragma unroll
        for (int i = 0; i < kMoved; ++i)
            if (base + i * threads < all) *to[i] = move_codes(w[i], by);
    }
}

// The largest magnitude among finite values. (fmaxf passes NaN over.)
template <int N>
__device__ __forceinline__ float largest_finite(const float (&x)[N], const float (&y)[N]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, fmaxf(fabsf(x[j]), fabsf(y[j])));
    if (m == INFINITY) {
        m = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (fabsf(x[j]) < INFINITY) m = fmaxf(m, fabsf(x[j]));
            if (fabsf(y[j]) < INFINITY) m = fmaxf(m, fabsf(y[j]));
        }
    }
    return m;
}

// Codes of values times `inv`.
template <int N>
__device__ __forceinline__ void store_codes(unsigned char* to, const float (&f)[N], float inv) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = f[i] * inv;
    if constexpr (N == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16,
                                                   e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    else if constexpr (N == 4)
        *reinterpret_cast<uint32_t*>(to) = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    else
        *to = static_cast<unsigned char>(e4m3x2(x[0], 0.f));
}

// The smallest power of two that is at least `scale` (positive, finite), 2^127 where there is none in FP32.
__device__ __forceinline__ float power_above(float scale) {
    const uint32_t bits = __float_as_uint(scale);
    const uint32_t up = (bits & 0x7fffffu) != 0u ? (bits & 0x7f800000u) + 0x800000u : bits;
    return fminf(__uint_as_float(up), 0x1p127f);
}
// One over a power of two from 2^-126 on. (That of 2^127 is subnormal.)
__device__ __forceinline__ float one_over(float power) {
    return power < 0x1p127f ? __uint_as_float((254u << 23) - __float_as_uint(power)) : 0x1p-127f;
}
// Whether the codes of a block move when its scale does: it grows, or comes down to the largest power of two.
__device__ __forceinline__ bool scale_moves(float old, float scale) { return scale > old || old > 0x1p127f; }

// The smallest power of two that is at least top / 448, no smaller than 2^-30; `top`: bits of a finite FP32 >= 0.
__device__ __forceinline__ float scale_for(uint32_t top) {
    // top = m 2^e with 1 <= m < 2; 448 = 1.75 * 2^8. (A subnormal's exponent reads as one below: under the floor.)
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -30) + 127) << 23);
}

// A lane's groups of a run's rows (64 values), kept in shared memory as they come: no other lane reads them. The copies
// are asynchronous, so that what is in flight takes no registers.
template <int VEC>
constexpr int kLineBytes = VEC == 1 ? 256 : 1024;                    // of a warp's groups: 32 lanes of one group each

__device__ __forceinline__ void copy_async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_addr(to)), "l"(from) : "memory");
}
template <int VEC, bool F32>
__device__ __forceinline__ void keep_group(unsigned char* line, int lane, const char* row, int c0, int c1) {
    constexpr int es = F32 ? 4 : 2;
    if constexpr (VEC > 1) {
        copy_async16(line + lane * 16, row + c0 * es);
        copy_async16(line + 512 + lane * 16, row + c1 * es);
    } else {
        Cols<1, F32> a, b;
        a.load(row, c0);
        b.load(row, c1);
        *reinterpret_cast<uint2*>(line + lane * 8) = make_uint2(a.w[0], b.w[0]);
    }
}
template <int VEC, bool F32>
__device__ __forceinline__ void kept_group(const unsigned char* line, int lane, float (&x)[VEC], float (&y)[VEC]) {
    Cols<VEC, F32> a, b;
    if constexpr (VEC > 1) {
        a.load(reinterpret_cast<const char*>(line + lane * 16), 0);
        b.load(reinterpret_cast<const char*>(line + 512 + lane * 16), 0);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(line + lane * 8);
        a.w[0] = v.x;
        b.w[0] = v.y;
    }
    a.values(x);
    b.values(y);
}

__device__ __forceinline__ void keep_turned(unsigned char* line, int lane, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<float4*>(line + lane * 16) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(line + 512 + lane * 16) = make_float4(y[0], y[1], y[2], y[3]);
}

// Threads of a team's warps wait for each other.
__device__ __forceinline__ void team_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// Single tokens, as a decode step brings them: the lanes of a token's head are a team of their own, as many of them in a
// warp as it has room for, with the row in registers and its sines computed by the lanes that need them. runs, held, code_at
// and scale_at: see write_blocks.
template <int VEC, bool F32>
__device__ __forceinline__ void write_singles(const RopeParams& p, const BlockScales& b, const AppendShape& a, int64_t first,
                                              bool is_k, int share, int shares, uint32_t runs, int held, int64_t code_at,
                                              int64_t scale_at) {
    constexpr int es = F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = a.groups, half = p.rot_dim / 2;
    const int sub = lane / groups, gi = lane - sub * groups;
    const bool split = gi * VEC < half && !p.interleaved;
    const int c0 = split ? gi * VEC : gi * 2 * VEC, c1 = split ? half + gi * VEC : gi * 2 * VEC + VEC;
    const int64_t stride = (is_k ? p.k_stride : p.v_stride) * es;
    const char* const rows = static_cast<const char*>(is_k ? p.k : p.v) + first * stride;
    const int items = __popc(runs) * p.kv_heads, before = __popc(runs & ((1u << lane) - 1u));
#pragma unroll 1
    for (int base = (share * kAppendWarps + warp) * a.across; base < items; base += shares * kAppendWarps * a.across) {
        const int item = base + sub;
        const int ri = p.kv_heads == 1 ? item : static_cast<int>(__umulhi(static_cast<uint32_t>(item), a.per_head));
        const int head = item - ri * p.kv_heads;
        const bool live = sub < a.across && item < items;
        // The lane of the item's run: the one with `ri` of them before it.
        int run = 0;
        for (uint32_t rest = __ballot_sync(0xffffffffu, runs >> lane & 1u); rest; rest &= rest - 1) {
            const int at = __ffs(rest) - 1;
            if (__shfl_sync(0xffffffffu, before, at) == ri) run = at;
        }
        const int held_run = __shfl_sync(0xffffffffu, held, run);
        const int64_t code_run = __shfl_sync(0xffffffffu, code_at, run), scale_run = __shfl_sync(0xffffffffu, scale_at, run);
        float x[VEC], y[VEC];
        float* const scale_to = (is_k ? b.k : b.v) + scale_run + head * b.head_stride;
        unsigned char* const to = (is_k ? p.kc : p.vc) + code_run + head * p.head_stride;
        unsigned char* const block_at = to - held_run * p.slot_stride;
        float old = 0.f;
        uint32_t top = 0;
        if (live) {
            Cols<VEC, F32> u, v;
            u.load(rows + run * stride + head * p.head_dim * es, c0);
            v.load(rows + run * stride + head * p.head_dim * es, c1);
            if (held_run > 0) old = *scale_to;
            float cs[VEC], sn[VEC];
            const bool turned = is_k && gi * VEC < half;
            if (turned) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int pair = gi * VEC + j;
                    const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
                    const int32_t pos = p.positions[axis * p.axis_stride + first + run];
                    const float2 of = turn_of(pos, static_cast<uint64_t>(p.freqs[pair]));
                    cs[j] = of.x;
                    sn[j] = of.y;
                }
            }
            u.values(x);
            v.values(y);
            if (turned) turn_group<VEC>(x, y, p.interleaved, cs, sn);
            top = __float_as_uint(largest_finite<VEC>(x, y));
        }
        // The largest value of the team's lanes: of those behind in the row, then the first one's for all.
        for (int o = 1; o < groups; o <<= 1) {
            const uint32_t other = __shfl_down_sync(0xffffffffu, top, o);
            if (gi + o < groups) top = max(top, other);
        }
        top = __shfl_sync(0xffffffffu, top, min(sub * groups, 31));
        const float need = scale_for(top);
        const float scale = held_run > 0 ? fmaxf(power_above(old), need) : need;
        const float inv = one_over(scale);
        // Earlier tokens move to the new scale: the whole warp for each team whose scale changes.
        const uint32_t grown = __ballot_sync(0xffffffffu, live && gi == 0 && held_run > 0 && scale_moves(old, scale));
        for (uint32_t rest = grown; rest; rest &= rest - 1) {
            const int at = __ffs(rest) - 1;
            unsigned char* const block =
                reinterpret_cast<unsigned char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(block_at), at));
            move_block(block, p.slot_stride, __shfl_sync(0xffffffffu, held_run, at), p.head_dim,
                       __shfl_sync(0xffffffffu, old * inv, at), lane, 32);
        }
        if (!live) continue;
        if (gi == 0 && scale != old) *scale_to = scale;              // (every lane has the old one)
        store_codes<VEC>(to + c0, x, inv);
        store_codes<VEC>(to + c1, y, inv);
    }
}

// NI: groups that a lane keeps.
template <int VEC, bool F32, int NI>
__device__ __forceinline__ void write_blocks(const RopeParams& p, const BlockScales& b, const AppendShape& a, int cta) {
    constexpr int es = F32 ? 4 : 2;
    constexpr bool kTurnOnce = F32 && VEC > 1;                       // turned rows have room where they were
    extern __shared__ __align__(16) unsigned char s_rows[];          // every warp's lines; then
    float* const s_cos = reinterpret_cast<float*>(s_rows + kAppendWarps * NI * kLineBytes<VEC>);   // [token][pair], and sines
    float* const s_sin = s_cos + a.turns;
    __shared__ uint32_t s_top[2][kAppendWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char* const lines = s_rows + warp * NI * kLineBytes<VEC>;
    const int win = a.kv_shift >= 0 ? cta >> a.kv_shift : cta / a.kv_parts;
    const int part = cta - win * a.kv_parts, shares = a.kv_parts >> 1;
    const bool is_k = part < shares;                                 // the others take v
    const int share = is_k ? part : part - shares;
    const int64_t first = static_cast<int64_t>(win) * a.window;
    const int half = p.rot_dim / 2, groups = a.groups;

    // The runs of the window: every warp finds them by itself, lane i the one that begins at token `first + i`. The bits
    // of goes_on: tokens that go on in the block of the one before them.
    int n = 0, held = 0;                                             // its tokens; earlier tokens of the block
    int64_t code_at = 0, scale_at = 0;                               // the first token's codes and the scale, head 0
    uint32_t runs;
    {
        uint32_t goes_on[3];
        int slot = -1;
        const int reach = a.window - 1 + b.tokens;                   // no run of the window goes further
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            goes_on[x] = 0u;
            if (x * 32 >= reach) continue;
            const int j = x * 32 + lane;
            bool on = false;
            if (j < reach && first + j < p.tokens) {
                const int mine = p.slots[first + j];
                const int before = first + j > 0 ? p.slots[first + j - 1] : -1;
                on = mine > 0 && before == mine - 1 && (b.shift >= 0 ? mine & (b.tokens - 1) : mine % b.tokens) != 0;
                if (x == 0) slot = mine;
            }
            goes_on[x] = __ballot_sync(0xffffffffu, on);
        }
        const bool begins = lane < a.window && slot >= 0 && slot < p.num_slots && !(goes_on[0] >> lane & 1u);
        runs = __ballot_sync(0xffffffffu, begins);
        if (begins) {
            const uint64_t low = goes_on[0] | static_cast<uint64_t>(goes_on[1]) << 32;
            const uint64_t after = low >> (lane + 1) | static_cast<uint64_t>(goes_on[2]) << (63 - lane);
            n = __ffsll(static_cast<long long>(~after));             // one more than the tokens that go on
            if (n == 0) n = 64;
            const int page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
            const int place = slot - page * p.page_size;
            const int blk = b.shift >= 0 ? place >> b.shift : place / b.tokens;
            held = place - blk * b.tokens;
            code_at = page * p.page_stride + place * p.slot_stride;
            scale_at = page * b.page_stride + blk * b.block_stride;
        }
    }
    const int longest = __reduce_max_sync(0xffffffffu, n);
    if constexpr (VEC > 1) {
        if (longest <= 1) {
            write_singles<VEC, F32>(p, b, a, first, is_k, share, shares, runs, held, code_at, scale_at);
            return;
        }
    }
    // Warps of a team: 1, 2, 4 or 8.
    const int slices = (longest + a.tokens_held - 1) / a.tokens_held;
    const int team_shift = slices <= 1 ? 0 : slices <= 2 ? 1 : slices <= 4 ? 2 : 3;
    const int team = warp >> team_shift, rank = warp & ((1 << team_shift) - 1), at_once = kAppendWarps >> team_shift;
    const int items = __popc(runs) * p.kv_heads;                     // runs and heads
    if (share * at_once >= items) return;

    // A lane's groups: the same group of every `across`-th token of the warp's (where groups are pairs, the groups of all
    // tokens one after the other).
    const int sub = VEC > 1 ? lane / groups : 0;
    const bool in_row = VEC == 1 || sub < a.across;
    const int tk0 = rank * (VEC > 1 ? NI * a.across : 0) + sub, gi0 = VEC > 1 ? lane - sub * groups : 0;
    auto group_at = [&](int i, int& tk, int& gi) {
        if constexpr (VEC > 1) {
            tk = tk0 + i * a.across;
            gi = gi0;
        } else {
            const int u = (rank * NI + i) * 32 + lane;
            tk = groups == 1 ? u : static_cast<int>(__umulhi(static_cast<uint32_t>(u), a.per_group));
            gi = u - tk * groups;
        }
    };
    auto columns_of = [&](int gi, int& c0, int& c1) {
        const bool split = gi * VEC < half && !p.interleaved;
        c0 = split ? gi * VEC : gi * 2 * VEC;
        c1 = split ? half + gi * VEC : gi * 2 * VEC + VEC;
    };
    const int64_t stride = (is_k ? p.k_stride : p.v_stride) * es;
    const char* const rows = static_cast<const char*>(is_k ? p.k : p.v) + first * stride;
    // The head and the run (its first token, from the window's on) of the team's item.
    int item = share * at_once + team, head = 0, run = 0, n_run = 0;
    auto locate = [&]() {
        const int ri = p.kv_heads == 1 ? item : static_cast<int>(__umulhi(static_cast<uint32_t>(item), a.per_head));
        head = item - ri * p.kv_heads;
        run = __ffs(__ballot_sync(0xffffffffu, (runs >> lane & 1u) && __popc(runs & ((1u << lane) - 1u)) == ri)) - 1;
        n_run = __shfl_sync(0xffffffffu, n, run);
    };
    auto fetch = [&]() {
        int tk, gi, c0, c1;
        group_at(0, tk, gi);
        columns_of(gi, c0, c1);
        const char* row = rows + (run + tk) * stride + head * p.head_dim * es;
#pragma unroll 4
        for (int i = 0; i < NI; ++i) {
            if constexpr (VEC == 1) {
                group_at(i, tk, gi);
                columns_of(gi, c0, c1);
                row = rows + (run + tk) * stride + head * p.head_dim * es;
            }
            if (in_row && tk < n_run) keep_group<VEC, F32>(lines + i * kLineBytes<VEC>, lane, row, c0, c1);
            if constexpr (VEC > 1) {
                tk += a.across;
                row += a.across * stride;
            }
        }
    };
    if (item < items) {
        locate();
        fetch();
    }
    const int table0 = __ffs(runs) - 1;                              // the first token of the table of sines
    if (is_k) {
        const int end = __reduce_max_sync(0xffffffffu, n > 0 ? lane + n : 0);
        const int dt = kAppendThreads / half, dp = kAppendThreads - dt * half;
        int t = tid / half, pair = tid - t * half, to = tid;
        t += table0;
        constexpr int U = 4;                                         // at a time, so that their loads are
        if (dp == 0) {                                               // the same pair again and again
            const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
            const uint64_t freq = static_cast<uint64_t>(p.freqs[pair]);
            const int32_t* const at = p.positions + axis * p.axis_stride + first;
            for (; t < end; t += U * dt) {
                int32_t pos[U];
#pragma unroll
                for (int i = 0; i < U; ++i) pos[i] = at[min(t + i * dt, end - 1)];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const float2 cs = turn_of(pos[i], freq);
                    if (t + i * dt < end) {
                        s_cos[to + i * kAppendThreads] = cs.x;
                        s_sin[to + i * kAppendThreads] = cs.y;
                    }
                }
                to += U * kAppendThreads;
            }
        }
        while (t < end) {
            int32_t pos[U];
            uint64_t freq[U];
            bool in[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                in[i] = t < end;
                const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
                pos[i] = p.positions[axis * p.axis_stride + first + (in[i] ? t : end - 1)];
                freq[i] = static_cast<uint64_t>(p.freqs[pair]);
                t += dt;
                pair += dp;
                if (pair >= half) {
                    pair -= half;
                    ++t;
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float2 cs = turn_of(pos[i], freq[i]);
                if (in[i]) {
                    s_cos[to] = cs.x;
                    s_sin[to] = cs.y;
                }
                to += kAppendThreads;
            }
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int round = 0; item < items; ++round) {
        const int held_run = __shfl_sync(0xffffffffu, held, run);
        const int64_t code_run = __shfl_sync(0xffffffffu, code_at, run), scale_run = __shfl_sync(0xffffffffu, scale_at, run);
        float* const scale_to = (is_k ? b.k : b.v) + scale_run + head * b.head_stride;
        const float old = held_run > 0 ? *scale_to : 0.f;
        asm volatile("cp.async.wait_all;" ::: "memory");
        // Group i of this lane, turned.
        auto turned = [&](int i, int tk, int gi, float (&x)[VEC], float (&y)[VEC]) {
            kept_group<VEC, F32>(lines + i * kLineBytes<VEC>, lane, x, y);
            if (is_k && gi * VEC < half) {
                const int at = (run - table0 + tk) * half + gi * VEC;
                float cs[VEC], sn[VEC];
                load_floats<VEC>(s_cos + at, cs);
                load_floats<VEC>(s_sin + at, sn);
                turn_group<VEC>(x, y, p.interleaved, cs, sn);
            }
        };
        float most = 0.f;                                            // of the finite values (fmaxf passes NaN over)
#pragma unroll 2
        for (int i = 0; i < NI; ++i) {
            int tk, gi;
            group_at(i, tk, gi);
            if (!in_row || tk >= n_run) continue;
            float x[VEC], y[VEC];
            turned(i, tk, gi, x, y);
            if constexpr (kTurnOnce)
                if (is_k) keep_turned(lines + i * kLineBytes<VEC>, lane, x, y);
            most = fmaxf(most, largest_finite<VEC>(x, y));
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
        if (team_shift > 0) {
            if (lane == 0) s_top[round & 1][warp] = top;
            team_barrier(1 + team, 32 << team_shift);
            top = __reduce_max_sync(0xffffffffu, s_top[round & 1][(warp - rank) | (lane & ((1 << team_shift) - 1))]);
        }
        const float need = scale_for(top);
        const float scale = held_run > 0 ? fmaxf(power_above(old), need) : need;
        const float inv = one_over(scale);
        unsigned char* const block_at = (is_k ? p.kc : p.vc) + code_run + head * p.head_stride - held_run * p.slot_stride;
        if (held_run > 0 && scale_moves(old, scale)) {               // earlier tokens move to the new scale
            move_block(block_at, p.slot_stride, held_run, p.head_dim, old * inv, rank * 32 + lane, 32 << team_shift);
        }
        if (rank == 0 && lane == 0 && scale != old) *scale_to = scale;   // (every lane has the old one)
        {
            int tk, gi, c0, c1;
            group_at(0, tk, gi);
            columns_of(gi, c0, c1);
            unsigned char* to = block_at + (held_run + tk) * p.slot_stride;
#pragma unroll 2
            for (int i = 0; i < NI; ++i) {
                if constexpr (VEC == 1) {
                    group_at(i, tk, gi);
                    columns_of(gi, c0, c1);
                    to = block_at + (held_run + tk) * p.slot_stride;
                }
                if (in_row && tk < n_run) {
                    float x[VEC], y[VEC];
                    if constexpr (kTurnOnce) kept_group<VEC, F32>(lines + i * kLineBytes<VEC>, lane, x, y);
                    else turned(i, tk, gi, x, y);
                    store_codes<VEC>(to + c0, x, inv);
                    store_codes<VEC>(to + c1, y, inv);
                }
                if constexpr (VEC > 1) {
                    tk += a.across;
                    to += a.across * p.slot_stride;
                }
            }
        }
        item += shares * at_once;
        if (item < items) {
            locate();
            fetch();
        }
    }
}

// The queries of TT tokens, `visit` heads a CTA: as gemv_rope turns them.
template <int VEC, bool F32, int TT>
__device__ __forceinline__ void turn_queries(const RopeParams& p, const AppendShape& a, int64_t tok0, int part) {
    constexpr int GAP = VEC > 1 ? 2 : 0;                             // a warp's groups lie in different banks
    __shared__ __align__(16) float2 s_turn[TT][GEMV_MAX_HEAD_DIM / 2 / VEC * (VEC + GAP)];
    constexpr int es = F32 ? 4 : 2;
    const int groups = a.groups, half = p.rot_dim / 2;
    const int hy = groups == 1 ? threadIdx.x : __umulhi(threadIdx.x, a.per_group), gi = threadIdx.x - hy * groups;
    const int h = part * a.visit + hy;
    const bool is_head = hy < a.visit && h < p.q_heads;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TT), p.tokens - tok0));
    const bool turned = gi * VEC < half;
    const int c0 = turned && !p.interleaved ? gi * VEC : gi * 2 * VEC;
    const int c1 = turned && !p.interleaved ? half + gi * VEC : gi * 2 * VEC + VEC;
    Cols<VEC, F32> u[TT], v[TT];
    int slot[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        if (is_head && i < tokens) {
            const char* const row = static_cast<const char*>(p.q) + ((tok0 + i) * p.q_stride + h * p.head_dim) * es;
            u[i].load(row, c0);
            v[i].load(row, c1);
        }
        slot[i] = i < tokens ? p.slots[tok0 + i] : -1;
    }
    for (int i = threadIdx.x; i < tokens * half; i += kAppendThreads) {
        int t = 0, pair = i;
#pragma unroll
        for (int x = 1; x < TT; ++x)
            if (pair >= half) {
                pair -= half;
                ++t;
            }
        const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
        s_turn[t][pair + pair / VEC * GAP] = turn_of(p.positions[axis * p.axis_stride + tok0 + t], p.freqs[pair]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        if (!is_head || slot[i] < 0 || slot[i] >= p.num_slots) continue;   // a padding row: nothing of it is written
        float x[VEC], y[VEC];
        u[i].values(x);
        v[i].values(y);
        if (turned) {
            float cs[VEC], sn[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float2 of = s_turn[i][gi * (VEC + GAP) + j];
                cs[j] = of.x;
                sn[j] = of.y;
            }
            turn_group<VEC>(x, y, p.interleaved, cs, sn);
        }
        uint16_t* const o = p.q_out + (tok0 + i) * p.q_out_stride + h * p.head_dim;
        store_bf16<VEC>(o, c0, x);
        store_bf16<VEC>(o, c1, y);
    }
}

// All but the last `left` groups of this thread's copies have landed. (A constant once the loop around it is unrolled.)
__device__ __forceinline__ void wait_copies(int left) {
    switch (left) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

// The same of kStreamTokens tokens, whose rows come by asynchronous copies to places of a thread's own: more in flight, less
// that begins and ends (4,051 tokens 29.3 -> 25.7 us; two tokens 26.9, eight 27.8).
template <int VEC, bool F32>
__device__ __forceinline__ void stream_queries(const RopeParams& p, const AppendShape& a, int64_t tok0, int part) {
    constexpr int GAP = 2, es = F32 ? 4 : 2, TT = kStreamTokens;
    extern __shared__ __align__(16) unsigned char s_rows[];
    float2* const s_turn = reinterpret_cast<float2*>(s_rows + TT * kAppendThreads * 32);
    const int groups = a.groups, half = p.rot_dim / 2, tid = threadIdx.x;
    const int pitch = half / VEC * (VEC + GAP);
    const int hy = groups == 1 ? tid : __umulhi(tid, a.per_group), gi = tid - hy * groups;
    const int h = part * a.visit + hy;
    const bool is_head = hy < a.visit && h < p.q_heads;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(TT), p.tokens - tok0));
    const bool turned = gi * VEC < half;
    const int c0 = turned && !p.interleaved ? gi * VEC : gi * 2 * VEC;
    const int c1 = turned && !p.interleaved ? half + gi * VEC : gi * 2 * VEC + VEC;
    unsigned char* const place = s_rows + tid * 16;
    {
        const char* row = static_cast<const char*>(p.q) + (tok0 * p.q_stride + h * p.head_dim) * es;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (is_head && i < tokens) {
                copy_async16(place + i * kAppendThreads * 32, row + c0 * es);
                copy_async16(place + i * kAppendThreads * 32 + kAppendThreads * 16, row + c1 * es);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            row += p.q_stride * es;
        }
    }
    const int lane = tid & 31;
    const int slots = lane < tokens ? p.slots[tok0 + lane] : -1;
    for (int i = tid; i < tokens * half; i += kAppendThreads) {
        int t = 0, pair = i;
#pragma unroll
        for (int x = 1; x < TT; ++x)
            if (pair >= half) {
                pair -= half;
                ++t;
            }
        const int axis = p.pair_axis ? min(max(p.pair_axis[pair], 0), p.axes - 1) : 0;
        s_turn[t * pitch + pair + pair / VEC * GAP] = turn_of(p.positions[axis * p.axis_stride + tok0 + t], p.freqs[pair]);
    }
    __syncthreads();
    uint16_t* o = p.q_out + tok0 * p.q_out_stride + h * p.head_dim;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        wait_copies(min(TT - 1 - i, 3));
        const int slot = __shfl_sync(0xffffffffu, slots, i);
        if (is_head && slot >= 0 && slot < p.num_slots) {            // else a padding row: nothing of it is written
            Cols<VEC, F32> u, v;
            u.load(reinterpret_cast<const char*>(place + i * kAppendThreads * 32), 0);
            v.load(reinterpret_cast<const char*>(place + i * kAppendThreads * 32 + kAppendThreads * 16), 0);
            float x[VEC], y[VEC];
            u.values(x);
            v.values(y);
            if (turned) {
                float cs[VEC], sn[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    const float4 of = *reinterpret_cast<const float4*>(&s_turn[i * pitch + gi * (VEC + GAP) + j]);
                    cs[j] = of.x; sn[j] = of.y; cs[j + 1] = of.z; sn[j + 1] = of.w;
                }
                turn_group<VEC>(x, y, p.interleaved, cs, sn);
            }
            store_bf16<VEC>(o, c0, x);
            store_bf16<VEC>(o, c1, y);
        }
        o += p.q_out_stride;
    }
}

template <int VEC, bool F32, int NI, int TT>
__global__ void __launch_bounds__(kAppendThreads, append_ctas(F32, TT))
append_blocks_kernel(const __grid_constant__ RopeParams p, const __grid_constant__ BlockScales b,
                     const __grid_constant__ AppendShape a) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    if (blockIdx.x < a.kv_ctas) {
        write_blocks<VEC, F32, NI>(p, b, a, static_cast<int>(blockIdx.x));
    } else {
        const unsigned q = blockIdx.x - a.kv_ctas;
        const unsigned at = a.parts_shift >= 0 ? q >> a.parts_shift : q / a.parts;
        const int64_t tok0 = static_cast<int64_t>(at) * TT;
        const int q_part = static_cast<int>(q - at * a.parts);
        if constexpr (TT == kStreamTokens) stream_queries<VEC, F32>(p, a, tok0, q_part);
        else turn_queries<VEC, F32, TT>(p, a, tok0, q_part);
    }
}

template <int VEC, bool F32, int NI, int TT>
cudaError_t launch_one(const RopeParams& p, const BlockScales& b, AppendShape a, cudaStream_t s, bool pdl) {
    const int64_t kv = (static_cast<int64_t>(p.tokens) + a.window - 1) / a.window * a.kv_parts;
    const int64_t q = (static_cast<int64_t>(p.tokens) + TT - 1) / TT * a.parts;
    if (kv + q > 0x7fffffff) return cudaErrorInvalidConfiguration;
    a.kv_ctas = static_cast<unsigned>(kv);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kv + q), 1, 1);
    cfg.blockDim = dim3(kAppendThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, append_blocks_kernel<VEC, F32, NI, TT>, p, b, a);
}

// log2 of a power of two, -1 of other numbers (254 single tokens 4.6 us with divisions, 4.4 with shifts).
int shift_of(int n) {
    int s = 0;
    while (1 << s < n) ++s;
    return 1 << s == n ? s : -1;
}

template <int VEC, bool F32, int NI>
cudaError_t launch_shape(const RopeParams& p, const BlockScales& b, int sm_count, cudaStream_t s, bool pdl) {
    AppendShape a = {};
    a.groups = p.head_dim / (2 * VEC);
    const int most = kAppendThreads / a.groups;                            // query heads of a CTA
    a.parts = (p.q_heads + most - 1) / most;
    a.parts_shift = shift_of(a.parts);
    a.visit = (p.q_heads + a.parts - 1) / a.parts;
    a.per_head = p.kv_heads > 1 ? static_cast<uint32_t>((uint64_t(1) << 32) / p.kv_heads + 1) : 0;
    a.per_group = a.groups > 1 ? static_cast<uint32_t>((uint64_t(1) << 32) / a.groups + 1) : 0;
    a.across = VEC > 1 ? 32 / a.groups : 1;
    a.tokens_held = VEC > 1 ? NI * a.across : std::max(1, NI * 32 / a.groups);
    // As many CTAs as take all heads of a whole block at once.
    const int slices = (b.tokens + a.tokens_held - 1) / a.tokens_held;
    const int at_once = kAppendWarps / (slices <= 1 ? 1 : slices <= 2 ? 2 : slices <= 4 ? 4 : 8);
    a.kv_parts = 2 * ((p.kv_heads + at_once - 1) / at_once);
    a.kv_shift = shift_of(a.kv_parts);
    // Windows as wide as it takes for one wave of CTAs, up to a block's tokens: a CTA without a run costs a microsecond
    // of its place, runs one after the other cost two each.
    // Queries by asynchronous copies where they are several waves of CTAs (us, registers -> so: 2,000 FP32 tokens of 32 heads
    // of 128 15.8 -> 14.3, 4,000 BF16 ones 19.8 -> 17.7; 1,021 FP32 8.3 -> 8.7, 2,000 BF16 11.2 -> 11.5).
    const int64_t queries = static_cast<int64_t>(p.tokens) * a.parts;
    const int tokens = VEC > 1 && queries >= 20 * sm_count ? kStreamTokens : queries >= 4 * sm_count ? kQueryTokens : 1;
    const int64_t wave = static_cast<int64_t>(append_ctas(F32, tokens)) * sm_count;
    const int64_t need = static_cast<int64_t>(p.tokens) * a.kv_parts;
    a.window = static_cast<int>(std::min<int64_t>({(need + wave - 1) / wave, std::max(b.tokens, 8), kMaxWindow}));
    a.turns = (a.window - 1 + b.tokens) * (p.rot_dim / 2);
    a.shared = kAppendWarps * NI * kLineBytes<VEC> + a.turns * 8;
    if constexpr (VEC > 1) {
        if (tokens == kStreamTokens) {
            a.shared = std::max(a.shared, kStreamTokens * (kAppendThreads * 32 + p.rot_dim / 2 / VEC * (VEC + 2) * 8));
            return launch_one<VEC, F32, NI, kStreamTokens>(p, b, a, s, pdl);
        }
    }
    return tokens > 1 ? launch_one<VEC, F32, NI, kQueryTokens>(p, b, a, s, pdl) : launch_one<VEC, F32, NI, 1>(p, b, a, s, pdl);
}

template <int VEC, bool F32, int NI, int TT>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(append_blocks_kernel<VEC, F32, NI, TT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kMostShared);
}

template <int VEC, bool F32, int NI>
cudaError_t prepare_shape() {
    cudaError_t e = prepare_one<VEC, F32, NI, 1>();
    if (e == cudaSuccess) e = prepare_one<VEC, F32, NI, kQueryTokens>();
    if constexpr (VEC > 1)
        if (e == cudaSuccess) e = prepare_one<VEC, F32, NI, kStreamTokens>();
    return e;
}

}  // namespace

cudaError_t prepare_append_blocks() {
    cudaError_t e = prepare_shape<8, false, 4>();
    if (e == cudaSuccess) e = prepare_shape<1, false, 32>();
    if (e == cudaSuccess) e = prepare_shape<1, true, 32>();
    if (e == cudaSuccess) e = prepare_shape<4, true, 4>();
    return e == cudaSuccess ? prepare_shape<4, true, 8>() : e;
}

cudaError_t launch_append_blocks(const RopeParams& p, const BlockScales& b, int sm_count, cudaStream_t s, bool pdl) {
    // Groups a lane keeps: 8 warps have to hold a block's tokens of a head. Four, which leave room for four CTAs an SM, do
    // but for FP32 heads of over 128 columns in blocks of over 32.
    if (!p.rows_f32)
        return p.vec >= 8 ? launch_shape<8, false, 4>(p, b, sm_count, s, pdl)
                          : launch_shape<1, false, 32>(p, b, sm_count, s, pdl);
    if (p.vec < 4) return launch_shape<1, true, 32>(p, b, sm_count, s, pdl);
    return kAppendWarps * 4 * (32 / (p.head_dim / 8)) >= b.tokens ? launch_shape<4, true, 4>(p, b, sm_count, s, pdl)
                                                                  : launch_shape<4, true, 8>(p, b, sm_count, s, pdl);
}

}  // namespace gemv
