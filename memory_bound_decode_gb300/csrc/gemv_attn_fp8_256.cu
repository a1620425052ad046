// Paged attention instances: FP8 cache, heads of up to 256 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(fp8_256, 256, true, false, 2)
}  // namespace gemv
