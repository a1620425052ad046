// Paged attention instances: BF16 cache, heads of up to 128 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(bf16_128, 128, false, false, 4)
}  // namespace gemv
