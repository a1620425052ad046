// Paged attention instances: BF16 cache, heads of up to 64 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(bf16_64, 64, false, 4)
}  // namespace gemv
