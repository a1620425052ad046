// Paged attention instances: BF16 cache, heads of up to 256 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(bf16_256, 256, false, false, 2)
}  // namespace gemv
