// Paged attention instances: FP8 cache with a scale for each block of tokens and head, heads of up to 128 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(fp8b_128, 128, true, true, 4)
}  // namespace gemv
