// Block tables and slot maps from request lengths.
//
// Two running sums over the requests (tokens, new pages) say where each
// request's tokens and pages begin; after them every token is on its own:
// its place in the request gives the page, from the request's table row or
// from the free list. One CTA does both where the tokens are few; otherwise a
// second kernel with a thread per token follows the first. Bound by latency:
// a few dependent reads and two block-wide sums.
#include <cstdint>
#include <cuda_runtime.h>

#include "gemv_attn_internal.h"

namespace gemv {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillTokens = 1024;        // tokens of one CTA of the second kernel
constexpr int kStartsMax = 4096;         // requests whose first tokens fit shared memory there
constexpr int64_t kOneCtaTokens = 8192;  // up to so many tokens the first kernel does it all

constexpr int64_t kMaxInt = 0x7fffffff;

enum { kServed = 0, kNoPages = 1, kTooLong = 2, kNoRoom = 3, kInvalid = 4 };

__host__ __device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One token of the step. first_of(r): the first token of request r, for r in 0..requests.
template <class First>
__device__ __forceinline__ void fill_token(const TablesParams& p, int64_t tok, int64_t total, First first_of) {
    int32_t slot = -1, position = 0;
    if (tok < total) {
        int lo = 0, hi = p.requests;                        // first_of(lo) <= tok < first_of(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first_of(mid) <= tok) lo = mid;
            else hi = mid;
        }
        if (p.status[lo] == kServed) {
            const int32_t count = p.new_tokens[lo];
            const int32_t old = p.new_lens[lo] - count;     // lens may be new_lens, already advanced
            position = old + static_cast<int32_t>(tok - first_of(lo));
            const int32_t blk = position / p.page_size, have = static_cast<int32_t>(ceil_div(old, p.page_size));
            int32_t page;
            if (blk >= have) {
                page = p.free_pages[p.page_start[lo] + (blk - have)];
                // the page's first token writes the table (every fresh page has one: it starts behind the old ones)
                if (position == blk * p.page_size) p.table[lo * p.table_stride + blk] = page;
            } else {
                page = p.table[lo * p.table_stride + blk];
            }
            if (page >= 0 && page < p.num_pages) slot = page * p.page_size + position - blk * p.page_size;
        }
    }
    p.slots[tok] = slot;
    p.positions[tok] = position;
}

// One CTA. FILL: also the tokens.
template <bool FILL>
__global__ void __launch_bounds__(kScanThreads) tables_scan_kernel(const __grid_constant__ TablesParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int64_t s_tok[32], s_page[32];
    __shared__ unsigned long long s_used;                   // pages taken: the largest running sum that was served
    __shared__ int32_t s_first[FILL ? kScanThreads : 1];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int64_t free_next = *p.free_next;
    const int64_t avail = free_next < 0 ? 0 : max(static_cast<int64_t>(p.free_cap) - free_next, int64_t(0));
    const int64_t row_tokens = static_cast<int64_t>(p.table_width) * p.page_size;
    int64_t tok_carry = 0, page_carry = 0;
    if (tid == 0) s_used = 0;
    __syncthreads();                                        // free_next has been read, s_used is zero
    for (int base = 0; base < p.requests; base += kScanThreads) {
        const int r = base + tid;
        const bool in = r < p.requests;
        const int64_t len = in ? p.lens[r] : 0, add = in ? p.new_tokens[r] : 0;
        const int64_t count = add < 0 ? 0 : add;
        int64_t tok_incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, tok_incl, o);
            if (lane >= o) tok_incl += up;
        }
        if (lane == 31) s_tok[w] = tok_incl;
        __syncthreads();
        int64_t tok_before = tok_carry, all = 0;
        {
            int64_t v = s_tok[lane];
            all = v;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            if (lane >= w) v = 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            tok_before += v;
        }
        tok_incl += tok_before;
        tok_carry += all;

        int state = kServed;
        if (len < 0 || add < 0) state = kInvalid;
        else if (len + add > row_tokens) state = kTooLong;
        else if (count > 0 && tok_incl > p.max_tokens) state = kNoRoom;
        const int64_t need =
            state == kServed ? ceil_div(len + count, p.page_size) - ceil_div(len, p.page_size) : 0;
        int64_t page_incl = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, page_incl, o);
            if (lane >= o) page_incl += up;
        }
        if (lane == 31) s_page[w] = page_incl;
        __syncthreads();
        {
            int64_t v = s_page[lane];
            all = v;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            if (lane >= w) v = 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            page_incl += v + page_carry;
        }
        page_carry += all;
        if (state == kServed && need > 0 && page_incl > avail) state = kNoPages;

        if (in) {
            const int64_t first = tok_incl - count;
            const int32_t first32 = static_cast<int32_t>(min(first, kMaxInt));
            p.token_start[r] = first32;
            if (FILL && p.requests <= kScanThreads) s_first[r] = first32;
            // Within the list where the request takes pages; where it takes none, never read.
            p.page_start[r] =
                state == kServed ? static_cast<int32_t>(min(free_next + page_incl - need, kMaxInt)) : -1;
            p.new_lens[r] = static_cast<int32_t>(state == kServed ? len + count : len);
            p.status[r] = state;
            if (state == kServed && need > 0) atomicMax(&s_used, static_cast<unsigned long long>(page_incl));
        }
        __syncthreads();                                    // s_tok and s_page have been read
    }
    if (tid == 0) {
        p.token_start[p.requests] = static_cast<int32_t>(min(tok_carry, kMaxInt));
        *p.free_next_out = static_cast<int32_t>(free_next + static_cast<int64_t>(s_used));
    }
    if constexpr (FILL) {
        __syncthreads();                                    // status, page_start and new_lens are written
        const bool near = p.requests <= kScanThreads;
        for (int64_t tok = tid; tok < p.max_tokens; tok += kScanThreads)
            fill_token(p, tok, tok_carry,
                       [&](int r) { return static_cast<int64_t>(near ? s_first[r] : p.token_start[r]); });
    }
}

__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const __grid_constant__ TablesParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ int32_t s_first[kStartsMax + 1];
    const bool near = p.requests <= kStartsMax;
    if (near)
        for (int r = threadIdx.x; r <= p.requests; r += kFillThreads) s_first[r] = p.token_start[r];
    __syncthreads();
    const int64_t total = p.token_start[p.requests];
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kFillTokens;
#pragma unroll
    for (int i = 0; i < kFillTokens / kFillThreads; ++i) {
        const int64_t tok = base + i * kFillThreads + threadIdx.x;
        if (tok < p.max_tokens)
            fill_token(p, tok, total,
                       [&](int r) { return static_cast<int64_t>(near ? s_first[r] : p.token_start[r]); });
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

cudaError_t launch_tables(const TablesParams& p, int /*sm_count*/, cudaStream_t s, bool pdl) {
    if (p.max_tokens <= kOneCtaTokens) return launch(tables_scan_kernel<true>, 1, kScanThreads, p, s, pdl);
    const cudaError_t e = launch(tables_scan_kernel<false>, 1, kScanThreads, p, s, pdl);
    if (e != cudaSuccess) return e;
    return launch(tables_fill_kernel, ceil_div(p.max_tokens, kFillTokens), kFillThreads, p, s, pdl);
}

}  // namespace gemv
