// Block tables and slot maps from request lengths.
//
// Two running sums over the requests (tokens, new pages) say where each
// request's tokens and pages begin; after them every token is on its own: its
// place in the request gives the page, from the request's row of the table or
// from the free list. Bound by latency: the lengths, a block-wide sum, a page
// number, its slot.
//
// Up to 1,024 requests one launch does it all. Every CTA sums all the requests
// for itself (cheaper than a second launch that waits for the first: half a
// million tokens of 509 requests took 13.5 us that way) and fills its share of
// the slots, four neighbouring tokens a thread (one at a time: 7.2 us; so:
// 5.9, against 0.65 for the bytes alone); the first one writes what belongs to
// the requests. In a decode step, where no request has more than a few tokens,
// a thread keeps its request and writes those tokens itself, with nothing to
// search (64 requests: 3.2 us, of which 2 are the launch). More requests, or
// many tokens with lens and new_lens the same array (which the first CTA then
// may not write while others read), take two launches.
#include <cstdint>
#include <cuda_runtime.h>

#include "gemv_attn_internal.h"
#include "gemv_common.cuh"

namespace gemv {
namespace {

constexpr int kTableThreads = 1024;      // and the requests of one launch
constexpr int kOneCtaTokens = 4096;      // up to so many tokens a single CTA takes them
constexpr int kFewTokens = 4;            // a request's tokens that its thread writes itself
constexpr int kRun = 4;                  // neighbouring tokens of a thread: one search, one 16-byte store
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 1024;        // tokens of a CTA of the second launch
constexpr int kStartsMax = 4096;         // requests whose first tokens fit shared memory there

constexpr uint32_t kMax = 0x7fffffffu;   // numbers stop here

enum { kServed = 0, kNoPages = 1, kTooLong = 2, kNoRoom = 3, kInvalid = 4 };

// a + b, at most kMax (both at most kMax). Adding so is associative.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kMax); }

__device__ __forceinline__ int blocks_of(const TablesParams& p, int len) {   // pages that len tokens take
    return p.page_shift >= 0 ? static_cast<int>((static_cast<uint32_t>(len) + p.page_size - 1) >> p.page_shift)
                             : len / p.page_size + (len % p.page_size != 0);
}
__device__ __forceinline__ int block_at(const TablesParams& p, int position) {
    return p.page_shift >= 0 ? position >> p.page_shift : position / p.page_size;
}

struct Request {
    int len, add;                        // as given
    int state;
    uint32_t first, page_first;          // tokens and new pages of the requests before it
};
struct Sums {
    uint32_t tokens, pages;              // of the requests so far
    uint32_t used;                       // pages taken
};

// The running sums over a chunk of requests, one per thread (`in`: there is one). `sums` holds those of the chunks
// before and then those up to this one's end. All threads call it.
__device__ __forceinline__ void sum_chunk(const TablesParams& p, Request& q, bool in, uint32_t avail, Sums& sums) {
    __shared__ uint32_t s_tok[32], s_page[32], s_used[32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t count = q.add > 0 ? q.add : 0;
    const int64_t end = static_cast<int64_t>(q.len) + q.add;
    q.state = !in || q.len < 0 || q.add < 0                                   ? kInvalid
              : end > static_cast<int64_t>(p.table_width) * p.page_size       ? kTooLong
                                                                              : kServed;
    uint32_t need = q.state == kServed ? blocks_of(p, q.len + q.add) - blocks_of(p, q.len) : 0;
    uint32_t tok_all, page_all;
    // Once; and once more where requests find no room for their tokens, and so take no pages.
    for (bool again = false;; again = true) {
        uint32_t tok = count, page = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, tok, o), b = __shfl_up_sync(0xffffffffu, page, o);
            if (lane >= o) {
                tok = sat_add(tok, a);
                page = sat_add(page, b);
            }
        }
        __syncthreads();                 // s_tok and s_page have been read
        if (lane == 31) {
            s_tok[w] = tok;
            s_page[w] = page;
        }
        uint32_t tok_ex = __shfl_up_sync(0xffffffffu, tok, 1), page_ex = __shfl_up_sync(0xffffffffu, page, 1);
        if (lane == 0) tok_ex = page_ex = 0;
        __syncthreads();
        uint32_t t = s_tok[lane], g = s_page[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, t, o), b = __shfl_up_sync(0xffffffffu, g, o);
            if (lane >= o) {
                t = sat_add(t, a);
                g = sat_add(g, b);
            }
        }
        tok_all = __shfl_sync(0xffffffffu, t, 31);
        page_all = __shfl_sync(0xffffffffu, g, 31);
        const uint32_t tw = __shfl_sync(0xffffffffu, t, max(w - 1, 0)), gw = __shfl_sync(0xffffffffu, g, max(w - 1, 0));
        q.first = sat_add(sums.tokens, sat_add(tok_ex, w > 0 ? tw : 0));
        q.page_first = sat_add(sums.pages, sat_add(page_ex, w > 0 ? gw : 0));
        if (again) break;
        // (In 64 bits: where max_tokens is kMax itself, a saturated sum would not be above it.)
        const bool over = q.state == kServed && count > 0 && static_cast<int64_t>(q.first) + count > p.max_tokens;
        if (over) {
            q.state = kNoRoom;
            need = 0;
        }
        if (!__syncthreads_or(over)) break;
    }
    const uint32_t pages = sat_add(q.page_first, need);
    if (q.state == kServed && need > 0 && (pages > avail || pages == kMax)) q.state = kNoPages;
    const uint32_t used = __reduce_max_sync(0xffffffffu, q.state == kServed && need > 0 ? pages : 0u);
    if (lane == 0) s_used[w] = used;
    __syncthreads();
    sums.used = max(sums.used, __reduce_max_sync(0xffffffffu, s_used[lane]));
    sums.tokens = sat_add(sums.tokens, tok_all);
    sums.pages = sat_add(sums.pages, page_all);
}

__device__ __forceinline__ uint32_t pages_left(const TablesParams& p, int free_next) {
    return free_next < 0 || free_next > p.free_cap ? 0u : static_cast<uint32_t>(p.free_cap - free_next);
}

// What belongs to request r (page_start: where its pages begin in the free list; never read where it takes none).
__device__ __forceinline__ void store_request(const TablesParams& p, int r, const Request& q, int free_next) {
    p.token_start[r] = static_cast<int32_t>(q.first);
    p.page_start[r] = q.state != kServed
                          ? -1
                          : static_cast<int32_t>(min(static_cast<int64_t>(free_next) + q.page_first, int64_t(kMax)));
    p.new_lens[r] = q.state == kServed ? q.len + q.add : q.len;
    p.status[r] = q.state;
}

// A token of a served request that had `old` tokens: its slot, and the table's entry if it is the first of a page (a
// page that is new this step has its first token in this step).
__device__ __forceinline__ void store_token(const TablesParams& p, int64_t tok, int r, int old, int position,
                                            int page_start) {
    const int blk = block_at(p, position), have = blocks_of(p, old), in = position - blk * p.page_size;
    int32_t* const entry = p.table + r * p.table_stride + blk;
    const int page = blk >= have ? p.free_pages[page_start + (blk - have)] : *entry;
    if (blk >= have && in == 0) *entry = page;
    p.slots[tok] = page >= 0 && page < p.num_pages ? page * p.page_size + in : -1;
    p.positions[tok] = position;
}
__device__ __forceinline__ void store_nothing(const TablesParams& p, int64_t tok) {
    p.slots[tok] = -1;
    p.positions[tok] = 0;
}

// The last request whose first token is not behind tok: that token's.
template <class First>
__device__ __forceinline__ int request_of(int requests, uint32_t tok, First first) {
    int lo = 0, hi = requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first(mid) <= tok) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Up to kTableThreads requests, any number of CTAs.
__global__ void __launch_bounds__(kTableThreads) tables_kernel(const __grid_constant__ TablesParams p) {
    __shared__ uint32_t s_first[kTableThreads];
    __shared__ int32_t s_old[kTableThreads], s_start[kTableThreads];   // s_old: -1 if the request was refused
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int r = threadIdx.x;
    const bool in = r < p.requests;
    const int free_next = *p.free_next;
    Request q = {in ? p.lens[r] : 0, in ? p.new_tokens[r] : 0};
    Sums sums = {};
    sum_chunk(p, q, in, pages_left(p, free_next), sums);
    if (blockIdx.x == 0) {
        if (in) store_request(p, r, q, free_next);
        if (r == 0) {
            p.token_start[p.requests] = static_cast<int32_t>(sums.tokens);
            *p.free_next_out = free_next + static_cast<int32_t>(sums.used);
        }
    }
    const int start = free_next + static_cast<int32_t>(q.page_first);
    if (gridDim.x == 1 && !__syncthreads_or(in && q.add > kFewTokens)) {
        if (in)
            for (int i = 0; i < q.add; ++i) {
                const int64_t tok = static_cast<int64_t>(q.first) + i;
                if (tok >= p.max_tokens) break;
                if (q.state == kServed) store_token(p, tok, r, q.len, q.len + i, start);
                else store_nothing(p, tok);
            }
        for (int64_t tok = sums.tokens + static_cast<int64_t>(r); tok < p.max_tokens; tok += kTableThreads)
            store_nothing(p, tok);
        return;
    }
    if (in) {
        s_first[r] = q.first;
        s_old[r] = q.state == kServed ? q.len : -1;
        s_start[r] = start;
    }
    __syncthreads();
    // Page numbers of a run are looked up together, then written together.
    const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kTableThreads * kRun;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kTableThreads + r) * kRun;
    for (int64_t tok = first; tok < p.max_tokens; tok += stride) {
        int of = request_of(p.requests, static_cast<uint32_t>(tok), [&](int i) { return s_first[i]; });
        int slot[kRun], position[kRun];
        const int32_t* from[kRun];
        int32_t* entry[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            while (of + 1 < p.requests && s_first[of + 1] <= static_cast<uint32_t>(tok + i)) ++of;
            from[i] = nullptr;
            entry[i] = nullptr;
            position[i] = 0;
            slot[i] = -1;
            const int old = s_old[of];
            if (tok + i >= min(static_cast<int64_t>(sums.tokens), p.max_tokens) || old < 0) continue;
            position[i] = old + static_cast<int>(tok + i - s_first[of]);
            const int blk = block_at(p, position[i]), have = blocks_of(p, old);
            slot[i] = position[i] - blk * p.page_size;
            int32_t* const at = p.table + of * p.table_stride + blk;
            from[i] = blk >= have ? p.free_pages + s_start[of] + (blk - have) : at;
            if (blk >= have && slot[i] == 0) entry[i] = at;
        }
        int page[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) page[i] = from[i] ? *from[i] : -1;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (entry[i]) *entry[i] = page[i];
            slot[i] = page[i] >= 0 && page[i] < p.num_pages ? page[i] * p.page_size + slot[i] : -1;
        }
        if (wide && tok + kRun <= p.max_tokens) {
            *reinterpret_cast<int4*>(p.slots + tok) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(p.positions + tok) = make_int4(position[0], position[1], position[2], position[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                if (tok + i < p.max_tokens) {
                    p.slots[tok + i] = slot[i];
                    p.positions[tok + i] = position[i];
                }
        }
    }
}

// Any number of requests: one CTA for the sums, then the tokens.
__global__ void __launch_bounds__(kTableThreads) tables_sums_kernel(const __grid_constant__ TablesParams p) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int free_next = *p.free_next;
    Sums sums = {};
    for (int base = 0; base < p.requests; base += kTableThreads) {
        const int r = base + threadIdx.x;
        const bool in = r < p.requests;
        Request q = {in ? p.lens[r] : 0, in ? p.new_tokens[r] : 0};
        sum_chunk(p, q, in, pages_left(p, free_next), sums);
        if (in) store_request(p, r, q, free_next);
    }
    if (threadIdx.x == 0) {              // behind sum_chunk's barriers: every thread has read free_next
        p.token_start[p.requests] = static_cast<int32_t>(sums.tokens);
        *p.free_next_out = free_next + static_cast<int32_t>(sums.used);
    }
}

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const __grid_constant__ TablesParams p) {
    __shared__ int32_t s_first[kStartsMax];
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const bool near = p.requests <= kStartsMax;
    if (near)
        for (int r = threadIdx.x; r < p.requests; r += kFillThreads) s_first[r] = p.token_start[r];
    __syncthreads();
    const int64_t total = p.token_start[p.requests];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kFillTokens;
#pragma unroll
    for (int i = 0; i < kFillTokens / kFillThreads; ++i) {
        const int64_t tok = base + i * kFillThreads + threadIdx.x;
        if (tok >= p.max_tokens) break;
        auto first = [&](int r) { return static_cast<uint32_t>(near ? s_first[r] : p.token_start[r]); };
        const int of = request_of(p.requests, static_cast<uint32_t>(tok), first);
        if (tok < total && p.status[of] == kServed) {
            const int old = p.new_lens[of] - p.new_tokens[of];       // lens may be new_lens, already advanced
            store_token(p, tok, of, old, old + static_cast<int>(tok - first(of)), p.page_start[of]);
        } else {
            store_nothing(p, tok);
        }
    }
}

cudaError_t launch(void (*f)(TablesParams), int64_t grid, int threads, const TablesParams& p, cudaStream_t s,
                   bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, f, p);
}

}  // namespace

cudaError_t launch_tables(const TablesParams& p, int sm_count, cudaStream_t s, bool pdl) {
    if (p.requests <= kTableThreads) {
        if (p.max_tokens <= kOneCtaTokens) return launch(tables_kernel, 1, kTableThreads, p, s, pdl);
        if (p.lens != p.new_lens && p.free_next != p.free_next_out) {
            const int64_t ctas = (p.max_tokens + kTableThreads * kRun - 1) / (kTableThreads * kRun);
            return launch(tables_kernel, ctas < sm_count ? ctas : sm_count, kTableThreads, p, s, pdl);
        }
    }
    const cudaError_t e = launch(tables_sums_kernel, 1, kTableThreads, p, s, pdl);
    if (e != cudaSuccess) return e;
    return launch(tables_fill_kernel, (p.max_tokens + kFillTokens - 1) / kFillTokens, kFillThreads, p, s, pdl);
}

}  // namespace gemv
