// Paged attention instances: FP8 cache, heads of up to 64 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(fp8_64, 64, true, 4)
}  // namespace gemv
