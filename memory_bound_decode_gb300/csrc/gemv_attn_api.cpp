// C-ABI front end of the decode step's attention half: argument checks and
// launches of the block tables, the rotary positions with the cache write, the
// paged decode attention, and the cache read back as rows.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether a pool of n items `stride` bytes apart stays within 2^60 bytes, so
// that the kernels' 64-bit offsets cannot wrap.
bool fits(int64_t n, int64_t stride) { return n <= 1 || stride <= (int64_t(1) << 60) / n; }

bool known_kind(int kind) {
    return kind == GEMV_CACHE_BF16 || kind == GEMV_CACHE_FP8 || kind == GEMV_CACHE_FP8_BLOCK;
}
// Elements of a 16-byte access.
int unit_of(int kind) { return kind == GEMV_CACHE_BF16 ? 8 : 16; }

// The fields of a cache with a scale for each block.
int check_block_scales(const gemv_kv_cache* c) {
    if (!c->k_block_scale || !c->v_block_scale || c->k_scale || c->v_scale) return GEMV_ERR_INVALID;
    if (c->block_tokens < 1 || c->block_tokens > GEMV_MAX_BLOCK_TOKENS || c->page_size % c->block_tokens != 0)
        return GEMV_ERR_INVALID;
    const int64_t n[3] = {c->num_pages, c->page_size / c->block_tokens, c->kv_heads};
    const int64_t st[3] = {c->scale_page_stride, c->scale_block_stride, c->scale_head_stride};
    for (int i = 0; i < 3; ++i)
        if (st[i] < (n[i] > 1) || st[i] > (int64_t(1) << 59) || !fits(n[i], 4 * st[i])) return GEMV_ERR_INVALID;
    if (!aligned(c->k_block_scale, 4) || !aligned(c->v_block_scale, 4)) return GEMV_ERR_ALIGN;
    return GEMV_OK;
}

int check_cache(const gemv_kv_cache* c) {
    if (!c || !c->k || !c->v) return GEMV_ERR_INVALID;
    if (!known_kind(c->kind)) return GEMV_ERR_INVALID;
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->kv_heads > 4096) return GEMV_ERR_INVALID;
    if (static_cast<int64_t>(c->num_pages) * c->page_size > 0x7fffffffLL) return GEMV_ERR_INVALID;
    const int unit = unit_of(c->kind);
    if (c->head_dim < unit || c->head_dim > GEMV_MAX_HEAD_DIM || c->head_dim % unit != 0) return GEMV_ERR_INVALID;
    const int64_t d = c->head_dim;
    const int64_t most = int64_t(1) << 59;                     // so that no product below can wrap
    if (c->page_stride > most || c->head_stride > most || c->slot_stride > most) return GEMV_ERR_INVALID;
    if ((c->num_pages > 1 && c->page_stride < d) || (c->kv_heads > 1 && c->head_stride < d) ||
        (c->page_size > 1 && c->slot_stride < d) || c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < 0)
        return GEMV_ERR_INVALID;
    if (!fits(c->num_pages, 2 * c->page_stride) || !fits(c->kv_heads, 2 * c->head_stride) ||
        !fits(c->page_size, 2 * c->slot_stride))
        return GEMV_ERR_INVALID;
    if (c->kind == GEMV_CACHE_BF16 && (c->k_scale || c->v_scale)) return GEMV_ERR_INVALID;
    if (c->page_stride % unit != 0 || c->head_stride % unit != 0 || c->slot_stride % unit != 0 || !aligned(c->k, 16) ||
        !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return GEMV_ERR_ALIGN;
    return c->kind == GEMV_CACHE_FP8_BLOCK ? check_block_scales(c) : GEMV_OK;
}

// log2 of a power of two, -1 of other sizes.
int shift_of(int32_t n) {
    if ((n & (n - 1)) != 0) return -1;
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

int elem_bytes(const gemv_kv_cache* c) { return c->kind == GEMV_CACHE_BF16 ? 2 : 1; }

int check_rope(const gemv_rope_args* a) {
    if (!a || !a->q || !a->k || !a->q_out || !a->positions || !a->freqs) return GEMV_ERR_INVALID;
    if (a->tokens < 0 || a->q_heads < 1 || a->q_heads > 4096 || a->kv_heads < 1 || a->kv_heads > 4096)
        return GEMV_ERR_INVALID;
    if (a->head_dim < 2 || a->head_dim > GEMV_MAX_HEAD_DIM || a->head_dim % 2 != 0) return GEMV_ERR_INVALID;
    if (a->rot_dim < 2 || a->rot_dim > a->head_dim || a->rot_dim % 2 != 0) return GEMV_ERR_INVALID;
    if (a->rows != GEMV_ROWS_F32 && a->rows != GEMV_ROWS_BF16) return GEMV_ERR_INVALID;
    if (a->pairs != GEMV_PAIRS_HALF && a->pairs != GEMV_PAIRS_INTERLEAVED) return GEMV_ERR_INVALID;
    if (a->axes < 1 || a->axes > GEMV_MAX_AXES || (a->axes > 1 && (!a->pair_axis || a->axis_stride < a->tokens)))
        return GEMV_ERR_INVALID;
    const int64_t qw = static_cast<int64_t>(a->q_heads) * a->head_dim;
    const int64_t kw = static_cast<int64_t>(a->kv_heads) * a->head_dim;
    if (a->q_stride < qw || a->k_stride < kw || a->q_out_stride < qw || (a->v && a->v_stride < kw))
        return GEMV_ERR_INVALID;
    const int64_t most = int64_t(1) << 40;                     // times 2^31 tokens at most
    if (a->q_stride > most || a->k_stride > most || a->q_out_stride > most || (a->v && a->v_stride > most) ||
        a->axis_stride > most)
        return GEMV_ERR_INVALID;
    const uintptr_t es = a->rows == GEMV_ROWS_F32 ? 4 : 2;
    if (!aligned(a->q, es) || !aligned(a->k, es) || !aligned(a->v, es) || !aligned(a->q_out, 2) ||
        !aligned(a->positions, 4) || !aligned(a->freqs, 8) || !aligned(a->pair_axis, 4))
        return GEMV_ERR_ALIGN;
    return GEMV_OK;
}

// What both rotary calls hand to the kernel.
void fill_rope(const gemv_rope_args* a, gemv::RopeParams* p) {
    p->q = a->q;
    p->k = a->k;
    p->positions = a->positions;
    p->freqs = a->freqs;
    p->pair_axis = a->axes > 1 ? a->pair_axis : nullptr;
    p->q_out = static_cast<uint16_t*>(a->q_out);
    p->q_stride = a->q_stride;
    p->k_stride = a->k_stride;
    p->v_stride = a->v_stride;
    p->q_out_stride = a->q_out_stride;
    p->axis_stride = a->axis_stride;
    p->tokens = a->tokens;
    p->q_heads = a->q_heads;
    p->kv_heads = a->kv_heads;
    p->head_dim = a->head_dim;
    p->rot_dim = a->rot_dim;
    p->rows_f32 = a->rows == GEMV_ROWS_F32;
    p->interleaved = a->pairs == GEMV_PAIRS_INTERLEAVED;
    p->axes = a->axes;
    // 16-byte reads (eight pairs of BF16 columns, four of FP32 ones) where every such group is whole and every row
    // starts on the boundary of its reads and writes; else a pair at a time.
    const int v = p->rows_f32 ? 4 : 8;
    const uintptr_t out = 2 * static_cast<uintptr_t>(v);
    p->vec = a->head_dim % (2 * v) == 0 && a->rot_dim % (2 * v) == 0 && a->q_stride % v == 0 && a->k_stride % v == 0 &&
                     a->q_out_stride % v == 0 && aligned(a->q, 16) && aligned(a->k, 16) && aligned(a->q_out, out) &&
                     (!a->v || (a->v_stride % v == 0 && aligned(a->v, 16)))
                 ? v
                 : 1;
}

int finish(cudaError_t e) { return e == cudaSuccess ? GEMV_OK : gemv::api_cuda_fail(e); }

}  // namespace

extern "C" {

int gemv_block_tables(const gemv_block_tables_args* a, void* stream) {
    if (!a || !a->lens || !a->new_tokens || !a->free_next || !a->table || !a->slots || !a->positions ||
        !a->token_start || !a->page_start || !a->new_lens || !a->status || !a->free_next_out)
        return GEMV_ERR_INVALID;
    // More requests than 2^30 would carry the kernels' 32-bit counts of them past 2^31 (the middle of a search, the
    // next chunk's first).
    if (a->requests < 1 || a->requests > (1 << 30) || a->page_size < 1 || a->num_pages < 1 || a->table_width < 1 ||
        a->free_cap < 0 || (a->free_cap > 0 && !a->free_pages))
        return GEMV_ERR_INVALID;
    if (static_cast<int64_t>(a->num_pages) * a->page_size > 0x7fffffffLL ||
        static_cast<int64_t>(a->table_width) * a->page_size > 0x7fffffffLL)
        return GEMV_ERR_INVALID;
    if (a->max_tokens < 1 || a->max_tokens > 0x7fffffffLL || a->table_stride < a->table_width ||
        a->table_stride > (int64_t(1) << 31))
        return GEMV_ERR_INVALID;
    const void* all[] = {a->lens, a->new_tokens, a->free_pages, a->free_next, a->table, a->slots, a->positions,
                         a->token_start, a->page_start, a->new_lens, a->status, a->free_next_out};
    for (const void* q : all)
        if (!aligned(q, 4)) return GEMV_ERR_ALIGN;
    int sm_count = 0;
    const int rc = gemv::api_device_state(&sm_count);
    if (rc != GEMV_OK) return rc;
    gemv::TablesParams p = {};
    p.lens = a->lens;
    p.new_tokens = a->new_tokens;
    p.free_pages = a->free_pages;
    p.free_next = a->free_next;
    p.table = a->table;
    p.slots = a->slots;
    p.positions = a->positions;
    p.token_start = a->token_start;
    p.page_start = a->page_start;
    p.new_lens = a->new_lens;
    p.status = a->status;
    p.free_next_out = a->free_next_out;
    p.table_stride = a->table_stride;
    p.max_tokens = a->max_tokens;
    p.requests = a->requests;
    p.page_size = a->page_size;
    p.num_pages = a->num_pages;
    p.table_width = a->table_width;
    p.free_cap = a->free_cap;
    p.page_shift = shift_of(a->page_size);
    return finish(gemv::launch_tables(p, sm_count, static_cast<cudaStream_t>(stream), gemv::api_pdl_enabled()));
}

int gemv_rope_freqs(const double* inv_freq, int n, int64_t* freqs) {
    if (!inv_freq || !freqs || n < 1) return GEMV_ERR_INVALID;
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(inv_freq[i])) return GEMV_ERR_INVALID;
    for (int i = 0; i < n; ++i) {
        // The fraction of a turn in [0, 1), as a multiple of 2^-64 (what rounds up to a whole turn wraps to 0).
        const double turns = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
        const double part = turns - std::floor(turns);
        const double high = std::floor(std::ldexp(part, 32));
        const double low = std::floor(std::ldexp(std::ldexp(part, 32) - high, 32));
        freqs[i] = static_cast<int64_t>((static_cast<uint64_t>(high) << 32) + static_cast<uint64_t>(low));
    }
    return GEMV_OK;
}

int gemv_rope(const gemv_rope_args* a, void* stream) {
    int rc = check_rope(a);
    if (rc != GEMV_OK) return rc;
    if (!a->k_out || a->v || a->slots) return GEMV_ERR_INVALID;
    if (a->k_out_stride < static_cast<int64_t>(a->kv_heads) * a->head_dim || a->k_out_stride > (int64_t(1) << 40))
        return GEMV_ERR_INVALID;
    if (!aligned(a->k_out, 2)) return GEMV_ERR_ALIGN;
    if (a->tokens == 0) return GEMV_OK;
    int sm_count = 0;
    if ((rc = gemv::api_device_state(&sm_count)) != GEMV_OK) return rc;
    gemv::RopeParams p = {};
    fill_rope(a, &p);
    if (a->k_out_stride % p.vec != 0 || !aligned(a->k_out, 2 * static_cast<uintptr_t>(p.vec))) p.vec = 1;
    p.kc = static_cast<unsigned char*>(a->k_out);           // a cache of pages of one token, token t in page t
    p.page_stride = a->k_out_stride * 2;
    p.head_stride = a->head_dim * 2;
    return finish(gemv::launch_rope(p, sm_count, static_cast<cudaStream_t>(stream), gemv::api_pdl_enabled()));
}

int gemv_rope_append(const gemv_rope_args* a, const gemv_kv_cache* c, void* stream) {
    int rc = check_rope(a);
    if (rc != GEMV_OK) return rc;
    if ((rc = check_cache(c)) != GEMV_OK) return rc;
    if (!a->v || !a->slots || a->k_out) return GEMV_ERR_INVALID;
    if (a->kv_heads != c->kv_heads || a->head_dim != c->head_dim) return GEMV_ERR_INVALID;
    if (!aligned(a->slots, 4)) return GEMV_ERR_ALIGN;
    if (a->tokens == 0) return GEMV_OK;
    int sm_count = 0;
    const bool blocks = c->kind == GEMV_CACHE_FP8_BLOCK;
    if ((rc = blocks ? gemv::api_cache_state(&sm_count) : gemv::api_device_state(&sm_count)) != GEMV_OK) return rc;
    gemv::RopeParams p = {};
    fill_rope(a, &p);
    p.v = a->v;
    p.slots = a->slots;
    p.kc = static_cast<unsigned char*>(c->k);
    p.vc = static_cast<unsigned char*>(c->v);
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    p.fp8 = c->kind == GEMV_CACHE_FP8;
    p.page_size = c->page_size;
    p.page_shift = shift_of(c->page_size);
    const int es = elem_bytes(c);
    p.page_stride = c->page_stride * es;
    p.head_stride = c->head_stride * es;
    p.slot_stride = c->slot_stride * es;
    p.num_slots = static_cast<int64_t>(c->num_pages) * c->page_size;
    if (blocks) {
        const gemv::BlockScales b = {c->k_block_scale, c->v_block_scale, c->scale_page_stride, c->scale_block_stride,
                                     c->scale_head_stride, c->block_tokens, shift_of(c->block_tokens)};
        return finish(gemv::launch_append_blocks(p, b, sm_count, static_cast<cudaStream_t>(stream),
                                                 gemv::api_pdl_enabled()));
    }
    return finish(gemv::launch_rope(p, sm_count, static_cast<cudaStream_t>(stream), gemv::api_pdl_enabled()));
}

int gemv_attn_query(int q_heads, int kv_heads, int head_dim, int kind, int sm_count, gemv_attn_info* out) {
    if (!out || sm_count < 1 || kv_heads < 1 || kv_heads > 4096 || q_heads < kv_heads || q_heads % kv_heads != 0)
        return GEMV_ERR_INVALID;
    if (!known_kind(kind)) return GEMV_ERR_INVALID;
    const int unit = unit_of(kind);
    if (head_dim < unit || head_dim > GEMV_MAX_HEAD_DIM || head_dim % unit != 0) return GEMV_ERR_INVALID;
    if (q_heads / kv_heads > gemv::kAttnMaxGroup) return GEMV_ERR_UNSUPPORTED;
    gemv::AttnLaunch l = {};
    const int rc = gemv::plan_attn(q_heads, kv_heads, head_dim, kind, sm_count, &l);
    if (rc != GEMV_OK) return rc;
    out->workspace_bytes = l.workspace_bytes;
    out->grid = l.grid;
    out->warps_per_cta = l.warps;
    out->head_tile = l.nb * 8;
    out->head_tiles = l.qtiles;
    out->dim_tile = l.dt;
    return GEMV_OK;
}

int gemv_attn_decode(const gemv_attn_args* a, const gemv_kv_cache* c, void* stream) {
    if (!a || !a->q || !a->out || !a->lens || !a->table || !a->workspace) return GEMV_ERR_INVALID;
    int rc = check_cache(c);
    if (rc != GEMV_OK) return rc;
    if (a->requests < 0 || a->q_heads < c->kv_heads || a->q_heads % c->kv_heads != 0) return GEMV_ERR_INVALID;
    const int group = a->q_heads / c->kv_heads;
    if (group > gemv::kAttnMaxGroup) return GEMV_ERR_UNSUPPORTED;
    const int64_t width = static_cast<int64_t>(a->q_heads) * c->head_dim;
    const int64_t most = int64_t(1) << 31;
    if (a->q_stride < width || a->out_stride < width || a->q_stride > most || a->out_stride > most)
        return GEMV_ERR_INVALID;
    if (a->table_width < 1 || a->table_stride < a->table_width || a->table_stride > most) return GEMV_ERR_INVALID;
    if (!std::isfinite(a->scale) || !std::isfinite(a->softcap) || a->softcap < 0.f || a->window < 0)
        return GEMV_ERR_INVALID;
    // The factors the kernel makes of them: an infinite one would turn a score of 0 into NaN.
    const float log2e = 1.4426950408889634f;
    if (!std::isfinite(a->softcap > 0.f ? a->scale / a->softcap : a->scale * log2e) ||
        !std::isfinite(a->softcap * log2e))
        return GEMV_ERR_INVALID;
    if (a->token_start && (a->rows < 0 || a->rows > 0x7fffffffLL)) return GEMV_ERR_INVALID;
    if (a->q_stride % 4 != 0 || a->out_stride % 4 != 0 || !aligned(a->q, 8) || !aligned(a->out, 8) ||
        !aligned(a->lse, 4) || !aligned(a->lens, 4) || !aligned(a->table, 4) || !aligned(a->token_start, 4) ||
        !aligned(a->status, 4) || !aligned(a->workspace, 16))
        return GEMV_ERR_ALIGN;
    // The kernel numbers the slices (16 tokens at least) of all rows in 31 bits.
    const int64_t reach = static_cast<int64_t>(a->table_width) * c->page_size;
    if (reach > 0x7fffff00LL || static_cast<double>(reach / 16 + 2) * a->requests * c->kv_heads > 0x7f000000)
        return GEMV_ERR_UNSUPPORTED;
    if (a->requests == 0) return GEMV_OK;
    gemv::AttnLaunch l = {};
    // What a GPU of one SM needs, so that a size left out is refused where there is none; then what this one needs.
    if ((rc = gemv::plan_attn(a->q_heads, c->kv_heads, c->head_dim, c->kind, 1, &l)) != GEMV_OK) return rc;
    if (a->workspace_bytes < l.workspace_bytes) return GEMV_ERR_INVALID;
    int sm_count = 0;
    if ((rc = gemv::api_attn_state(c->kind == GEMV_CACHE_FP8_BLOCK, &sm_count)) != GEMV_OK) return rc;
    if ((rc = gemv::plan_attn(a->q_heads, c->kv_heads, c->head_dim, c->kind, sm_count, &l)) != GEMV_OK) return rc;
    if (a->workspace_bytes < l.workspace_bytes) return GEMV_ERR_INVALID;
    gemv::AttnParams p = {};
    p.q = static_cast<const uint16_t*>(a->q);
    p.out = static_cast<uint16_t*>(a->out);
    p.lse = a->lse;
    p.lens = a->lens;
    p.token_start = a->token_start;
    p.status = a->status;
    p.rows = a->rows;
    p.table = a->table;
    p.kc = static_cast<const unsigned char*>(c->k);
    p.vc = static_cast<const unsigned char*>(c->v);
    p.k_scale = c->k_scale;
    p.v_scale = c->v_scale;
    char* ws = static_cast<char*>(a->workspace);
    p.ticket = reinterpret_cast<uint32_t*>(ws);
    p.part = reinterpret_cast<float*>(ws + gemv::kAttnTickets * 4);
    const int64_t heads = static_cast<int64_t>(l.grid) * l.nb * 8;
    p.part_warp = p.part + heads * 2 * l.dt;
    p.part_ml = p.part_warp + heads * gemv::kAttnWarps * l.dt;
    p.q_stride = a->q_stride;
    p.out_stride = a->out_stride;
    p.table_stride = a->table_stride;
    p.table_entries = gemv::attn_table_entries(a->requests, a->table_stride, a->table_width);
    p.page_stride = c->page_stride * elem_bytes(c);
    p.head_stride = c->head_stride * elem_bytes(c);
    p.slot_stride = c->slot_stride * elem_bytes(c);
    p.requests = a->requests;
    p.q_heads = a->q_heads;
    p.kv_heads = c->kv_heads;
    p.group = group;
    p.qtiles = l.qtiles;
    p.team_shift = l.team_shift;
    const int ctas = l.grid / l.qtiles >> l.team_shift;
    p.row_ctas = static_cast<int32_t>(ctas / (static_cast<int64_t>(a->requests) * (c->kv_heads >> l.team_shift)));
    p.cta_part = ctas > 1 ? ~uint64_t(0) / ctas + 1 : 0;      // 2^64 / ctas, rounded up
    p.quarter_of = (1u << 20) / (c->head_dim / 4) + 1;
    p.head_dim = c->head_dim;
    p.page_size = c->page_size;
    p.num_pages = c->num_pages;
    p.window = a->window;
    p.max_len = static_cast<int32_t>(reach);
    p.page_shift = shift_of(c->page_size);
    // Tensor copies where a box of at least 8 slots (the swizzle's pattern) divides page and slice.
    const int64_t es = elem_bytes(c);
    int rows = 1;
    while (rows < l.slice && c->page_size % (2 * rows) == 0) rows *= 2;
    if (rows >= 8 && gemv::api_on_current_device(c->k) && gemv::api_on_current_device(c->v)) {
        const int64_t dims[4] = {c->head_dim, c->page_size, c->kv_heads, c->num_pages};
        // The stride of a dimension of one entry is never used, but has to be a legal one.
        const int64_t st[3] = {c->page_size > 1 ? p.slot_stride : c->head_dim * es,
                               c->kv_heads > 1 ? p.head_stride : c->head_dim * es,
                               c->num_pages > 1 ? p.page_stride : c->head_dim * es};
        const int line = l.dt * es < 128 ? l.dt : static_cast<int>(128 / es);
        p.tma = gemv::api_encode_pool(&p.kmap, c->k, es == 1, dims, st, line, rows) &&
                gemv::api_encode_pool(&p.vmap, c->v, es == 1, dims, st, line, rows);
        p.box_shift = shift_of(rows);
    }
    if (c->kind == GEMV_CACHE_FP8_BLOCK) {
        p.k_block_scale = c->k_block_scale;
        p.v_block_scale = c->v_block_scale;
        p.scale_page_stride = c->scale_page_stride;
        p.scale_block_stride = c->scale_block_stride;
        p.scale_head_stride = c->scale_head_stride;
        p.block_tokens = c->block_tokens;
        p.block_shift = shift_of(c->block_tokens);
    }
    p.scale = a->scale;
    p.softcap = a->softcap;
    return finish(gemv::launch_attn(p, l, static_cast<cudaStream_t>(stream), gemv::api_pdl_enabled()));
}

int gemv_cache_read(const gemv_cache_read_args* a, const gemv_kv_cache* c, void* stream) {
    if (!a || !a->table || !a->row_start || (!a->k_out && !a->v_out)) return GEMV_ERR_INVALID;
    int rc = check_cache(c);
    if (rc != GEMV_OK) return rc;
    if (a->row_type != GEMV_ROWS_F32 && a->row_type != GEMV_ROWS_BF16) return GEMV_ERR_INVALID;
    if (a->requests < 0 || a->requests > (1 << 30) || a->rows < 0 || a->rows > 0x7fffffffLL) return GEMV_ERR_INVALID;
    const int64_t width = static_cast<int64_t>(c->kv_heads) * c->head_dim, most = int64_t(1) << 31;
    if (a->table_width < 1 || a->table_stride < a->table_width || a->table_stride > most) return GEMV_ERR_INVALID;
    if (static_cast<int64_t>(a->table_width) * c->page_size > 0x7fffffffLL) return GEMV_ERR_INVALID;
    if ((a->k_out && (a->k_out_stride < width || a->k_out_stride > most)) ||
        (a->v_out && (a->v_out_stride < width || a->v_out_stride > most)))
        return GEMV_ERR_INVALID;
    const int es = a->row_type == GEMV_ROWS_F32 ? 4 : 2, unit = 16 / es;
    if ((a->k_out && a->k_out_stride % unit != 0) || (a->v_out && a->v_out_stride % unit != 0) ||
        !aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !aligned(a->table, 4) || !aligned(a->begin, 4) ||
        !aligned(a->row_start, 4))
        return GEMV_ERR_ALIGN;
    if (a->requests == 0 || a->rows == 0) return GEMV_OK;
    int sm_count = 0;
    if ((rc = gemv::api_cache_state(&sm_count)) != GEMV_OK) return rc;
    gemv::ReadParams p = {};
    p.pool[0] = static_cast<const unsigned char*>(c->k);
    p.pool[1] = static_cast<const unsigned char*>(c->v);
    p.out[0] = static_cast<unsigned char*>(a->k_out);
    p.out[1] = static_cast<unsigned char*>(a->v_out);
    p.out_stride[0] = a->k_out_stride * es;
    p.out_stride[1] = a->v_out_stride * es;
    p.table = a->table;
    p.begin = a->begin;
    p.row_start = a->row_start;
    p.table_stride = a->table_stride;
    p.page_stride = c->page_stride * elem_bytes(c);
    p.head_stride = c->head_stride * elem_bytes(c);
    p.slot_stride = c->slot_stride * elem_bytes(c);
    p.rows = a->rows;
    p.requests = a->requests;
    p.table_width = a->table_width;
    p.num_pages = c->num_pages;
    p.page_size = c->page_size;
    p.page_shift = shift_of(c->page_size);
    p.kv_heads = c->kv_heads;
    p.head_dim = c->head_dim;
    p.fp8 = c->kind != GEMV_CACHE_BF16;
    p.rows_f32 = a->row_type == GEMV_ROWS_F32;
    // A scale per head is one for blocks of a page, the same in every page.
    p.block_tokens = c->page_size;
    p.block_shift = p.page_shift;
    if (c->kind == GEMV_CACHE_FP8_BLOCK) {
        p.scale[0] = c->k_block_scale;
        p.scale[1] = c->v_block_scale;
        p.scale_page_stride = c->scale_page_stride;
        p.scale_block_stride = c->scale_block_stride;
        p.scale_head_stride = c->scale_head_stride;
        p.block_tokens = c->block_tokens;
        p.block_shift = shift_of(c->block_tokens);
    } else {
        p.scale[0] = c->k_scale;
        p.scale[1] = c->v_scale;
        p.scale_head_stride = 1;
    }
    return finish(gemv::launch_read(p, static_cast<cudaStream_t>(stream), gemv::api_pdl_enabled()));
}

}  // extern "C"
