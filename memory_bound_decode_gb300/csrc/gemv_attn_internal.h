// Internal declarations of the decode step's attention half: block tables,
// rotary positions with the cache write, paged decode attention. Shared by
// their kernels and the C-ABI front end; the public interface is
// include/gemv.h.
#pragma once

#include <cstdint>
#include <cuda.h>   // CUtensorMap (the type only)
#include <cuda_runtime.h>

namespace gemv {

// ---- shared with gemv_api.cpp -------------------------------------------------
int api_device_state(int* sm_count);      // set-up of the current device; GEMV_OK or an error
int api_attn_state(bool block, int* sm_count);   // and of its attention kernels; block: with a scale for each block
int api_cache_state(int* sm_count);       // or of those that write a cache with scales for blocks and read a cache back
int api_cuda_fail(cudaError_t e);         // record e for gemv_last_cuda_error; GEMV_ERR_CUDA
bool api_pdl_enabled();
bool api_on_current_device(const void* p);   // whether p points into the current device's own memory
// A pool as a 4-D view (column, slot, head, page; strides in bytes) in boxes of
// `cols` columns x `rows` slots, swizzled; false if the driver rejects it.
bool api_encode_pool(CUtensorMap* map, const void* base, bool fp8, const int64_t (&dims)[4],
                     const int64_t (&strides)[3], int cols, int rows);

// ---- attention ----------------------------------------------------------------

constexpr int kAttnTickets = 1024;        // counters at the start of the workspace: rows, then groups of pieces
constexpr int kAttnMaxGroup = 1024;       // query heads per key-value head

constexpr int kAttnWarps = 8;
constexpr int kAttnRing = 16384;          // bytes of K and V in flight per warp

// Tokens a warp takes at a time: MMA tiles of 16 side by side hide each other's
// latency and share one reduction (BF16 at 128 columns: 9.3 TB/s of K and V
// with 16 tokens, 15.3 with 32, K and V from the L2). 64 with an FP8 cache and
// one block of heads, whose codes take longest to get through; 16 where the
// accumulators leave no registers, or the ring no room, for more. Without
// tensor copies a lane copies a token's rows: 32 at most.
// With a scale for each block, larger slices for groups of more than 8 heads too, as far as the registers go: 32 x 16,384
// tokens, 64 columns, groups of 16 heads 55.8 -> 44.4 us, of 32 heads 114.8 -> 83.0; 128 columns 67.2 -> 57.1 and
// 141.3 -> 115.9; 256 columns, 48 x 9,000 tokens, groups of 16 68.4 -> 54.5.
constexpr int attn_slice(int dt, int nb, bool fp8, bool tma, bool block = false) {
    if (block && nb > 1) return dt <= 128 && nb == 2 && tma ? 64 : 32;
    return (dt == 256 && (!fp8 || nb == 2)) || nb == 4 ? 16 : fp8 && nb == 1 && dt <= 128 && tma ? 64 : 32;
}

// Entries that a table of `width` per request, `stride` apart, reaches over:
// what lies behind the last row's is not the caller's to name.
constexpr int64_t attn_table_entries(int64_t requests, int64_t stride, int64_t width) {
    return requests > 0 ? (requests - 1) * stride + width : 0;
}

struct AttnParams {
    CUtensorMap kmap, vmap;     // views of the pools, if tma
    const uint16_t* q;          // BF16
    uint16_t* out;              // BF16
    float* lse;
    const int32_t* lens;
    const int32_t* token_start; // null: request r's query is row r
    const int32_t* status;      // null: none; not 0: the request was refused a place for its new tokens
    const int32_t* table;
    const unsigned char* kc;
    const unsigned char* vc;
    const float* k_scale;
    const float* v_scale;
    const float* k_block_scale; // a scale per block of tokens and head
    const float* v_block_scale;
    float* part;                // two pieces per CTA, of rows cut between CTAs: outputs,
    float* part_ml;             // maxima and sums
    float* part_warp;           // a piece per warp, of rows cut between a CTA's warps
    uint32_t* ticket;
    int64_t q_stride, out_stride, table_stride;
    int64_t table_entries;      // from the table's first to its last
    int64_t page_stride, head_stride, slot_stride;   // bytes
    int64_t scale_page_stride, scale_block_stride, scale_head_stride;   // elements
    int64_t rows;               // rows of q and out
    int32_t requests, q_heads, kv_heads, group, qtiles, team_shift;
    int32_t head_dim, page_size, num_pages, window, max_len;
    int32_t page_shift;         // log2 of page_size, -1 if it is no power of two
    int32_t block_tokens, block_shift;               // the same of a block with a scale
    int32_t tma;                // 1: tensor copies of 1 << box_shift slots
    int32_t box_shift;
    uint32_t quarter_of;        // x * quarter_of >> 20 is x / (head_dim / 4), up to 2,048
    uint64_t cta_part;          // the upper half of n * cta_part is n / teams, up to 2^31 (0: one team)
    int32_t row_ctas;           // CTAs for each row where all rows are of one length; 0: too many rows
    float scale, softcap;
};

struct AttnLaunch {
    int dt;            // head size the instance is built for: 64, 128 or 256
    int nb;            // blocks of 8 query heads a CTA carries
    int fp8;
    int block;         // a scale for each block of tokens and head
    int warps;
    int slice;         // tokens a warp takes at a time
    int qtiles, team_shift, grid;
    int64_t workspace_bytes;
};

int plan_attn(int q_heads, int kv_heads, int head_dim, int kind, int sm_count, AttnLaunch* l);   // kind: GEMV_CACHE_*

cudaError_t launch_attn(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl);
cudaError_t prepare_attn(bool block);     // the kernels over a cache with a scale for each block, or the others
cudaError_t read_attn_status(bool block, unsigned int* bits, bool reset);

// ---- rotary positions -----------------------------------------------------------

struct RopeParams {
    const void* q;
    const void* k;
    const void* v;              // null: no v
    const int32_t* positions;
    const int64_t* freqs;
    const int32_t* pair_axis;   // null: axis 0
    const int32_t* slots;       // null: k goes to row t of kc
    uint16_t* q_out;
    unsigned char* kc;          // the cache, or k_out
    unsigned char* vc;
    const float* k_scale;
    const float* v_scale;
    int64_t q_stride, k_stride, v_stride, q_out_stride;   // elements
    int64_t axis_stride;
    int64_t page_stride, head_stride, slot_stride;        // bytes
    int64_t num_slots;
    int32_t tokens, q_heads, kv_heads, head_dim, rot_dim, page_size;
    int32_t rows_f32, interleaved, fp8, axes, vec;
    int32_t page_shift;         // log2 of page_size, -1 if it is no power of two
};

cudaError_t launch_rope(const RopeParams& p, int sm_count, cudaStream_t s, bool pdl);

// The write into a cache with a scale for each block of tokens and head.
struct BlockScales {
    float* k;
    float* v;
    int64_t page_stride, block_stride, head_stride;       // elements
    int32_t tokens;             // of a block
    int32_t shift;              // its log2, -1 if it is no power of two
};

cudaError_t prepare_append_blocks();
cudaError_t launch_append_blocks(const RopeParams& p, const BlockScales& b, int sm_count, cudaStream_t s, bool pdl);

// ---- rows read back from a cache --------------------------------------------------

struct ReadParams {
    const unsigned char* pool[2];                         // k, v
    unsigned char* out[2];                                // null: not wanted
    const float* scale[2];      // per head, or of BlockScales' layout
    const int32_t* table;
    const int32_t* begin;       // null: 0
    const int32_t* row_start;
    int64_t table_stride;
    int64_t out_stride[2];                                // bytes
    int64_t page_stride, head_stride, slot_stride;        // bytes
    int64_t scale_page_stride, scale_block_stride, scale_head_stride;
    int64_t rows;
    int32_t requests, table_width, num_pages, page_size, kv_heads, head_dim;
    int32_t page_shift, block_tokens, block_shift;
    int32_t fp8, rows_f32;
};

cudaError_t prepare_read();
cudaError_t launch_read(const ReadParams& p, cudaStream_t s, bool pdl);
cudaError_t read_read_status(unsigned int* bits, bool reset);

// ---- block tables ---------------------------------------------------------------

struct TablesParams {
    const int32_t* lens;
    const int32_t* new_tokens;
    const int32_t* free_pages;
    const int32_t* free_next;
    int32_t* table;
    int32_t* slots;
    int32_t* positions;
    int32_t* token_start;
    int32_t* page_start;
    int32_t* new_lens;
    int32_t* status;
    int32_t* free_next_out;
    int64_t table_stride, max_tokens;
    int32_t requests, page_size, num_pages, table_width, free_cap;
    int32_t page_shift;         // log2 of page_size, -1 if it is no power of two
};

cudaError_t launch_tables(const TablesParams& p, int sm_count, cudaStream_t s, bool pdl);

}  // namespace gemv
