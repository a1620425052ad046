// Choice of the paged-attention instance, its grid and its workspace.
#include <algorithm>

#include "../../include/gemv.h"
#include "gemv_attn_internal.h"

namespace gemv {

#define GEMV_ATTN_DECL(SUFFIX)                                                                             \
    cudaError_t attn_prepare_##SUFFIX();                                                                   \
    cudaError_t attn_launch_##SUFFIX(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl); \
    cudaError_t attn_status_##SUFFIX(unsigned int* bits, bool reset);
GEMV_ATTN_DECL(bf16_64)
GEMV_ATTN_DECL(bf16_128)
GEMV_ATTN_DECL(bf16_256)
GEMV_ATTN_DECL(fp8_64)
GEMV_ATTN_DECL(fp8_128)
GEMV_ATTN_DECL(fp8_256)

// The instance of a shape: the smallest head size that holds head_dim, and as
// many blocks of 8 query heads as the group needs, up to what the output
// accumulators leave room for (32 heads; 16 where a head has over 128
// columns). A larger group is cut into tiles, one per CTA of a set of CTAs
// that read the same tokens at the same time. CTAs also form teams of 2, 4 or
// 8, as far as both the KV heads and the CTAs divide, a head of a block each.
int plan_attn(int q_heads, int kv_heads, int head_dim, int fp8, int sm_count, AttnLaunch* l) {
    const int group = q_heads / kv_heads;
    l->fp8 = fp8;
    l->dt = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    const int most = l->dt == 256 ? 2 : 4;
    const int blocks = (group + 7) / 8;
    l->nb = blocks <= 1 ? 1 : blocks <= 2 || most == 2 ? 2 : 4;
    l->qtiles = (blocks + l->nb - 1) / l->nb;
    l->grid = std::max(1, sm_count / l->qtiles) * l->qtiles;
    l->team_shift = 0;
    while (l->team_shift < 3 && ((kv_heads | l->grid / l->qtiles) >> l->team_shift & 1) == 0) ++l->team_shift;
    if (l->grid > kAttnTickets / 2) return GEMV_ERR_UNSUPPORTED;
    const int64_t heads = static_cast<int64_t>(l->grid) * (2 + kAttnWarps) * l->nb * 8;   // pieces of CTAs and warps
    l->workspace_bytes = kAttnTickets * 4 + heads * (2 + l->dt) * 4;
    l->warps = kAttnWarps;
    l->slice = attn_slice(l->dt, l->nb, fp8 != 0, true);
    return GEMV_OK;
}

cudaError_t launch_attn(const AttnParams& p, const AttnLaunch& l, cudaStream_t s, bool pdl) {
    if (l.fp8) {
        if (l.dt == 64) return attn_launch_fp8_64(p, l, s, pdl);
        if (l.dt == 128) return attn_launch_fp8_128(p, l, s, pdl);
        return attn_launch_fp8_256(p, l, s, pdl);
    }
    if (l.dt == 64) return attn_launch_bf16_64(p, l, s, pdl);
    if (l.dt == 128) return attn_launch_bf16_128(p, l, s, pdl);
    return attn_launch_bf16_256(p, l, s, pdl);
}

cudaError_t prepare_attn() {
    cudaError_t (*const all[])() = {attn_prepare_bf16_64, attn_prepare_bf16_128, attn_prepare_bf16_256,
                                    attn_prepare_fp8_64, attn_prepare_fp8_128, attn_prepare_fp8_256};
    for (auto f : all) {
        const cudaError_t e = f();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t read_attn_status(unsigned int* bits, bool reset) {
    cudaError_t (*const all[])(unsigned int*, bool) = {attn_status_bf16_64, attn_status_bf16_128,
                                                       attn_status_bf16_256, attn_status_fp8_64,
                                                       attn_status_fp8_128, attn_status_fp8_256};
    *bits = 0;
    for (auto f : all) {
        unsigned int b = 0;
        const cudaError_t e = f(&b, reset);
        if (e != cudaSuccess) return e;
        *bits |= b;
    }
    return cudaSuccess;
}

}  // namespace gemv
