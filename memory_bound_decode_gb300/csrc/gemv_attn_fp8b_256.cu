// Paged attention instances: FP8 cache with a scale for each block of tokens and head, heads of up to 256 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(fp8b_256, 256, true, true, 2)
}  // namespace gemv
