// Paged attention instances: FP8 cache, heads of up to 128 columns.
#include "gemv_attn_instances.cuh"

namespace gemv {
GEMV_ATTN_UNIT(fp8_128, 128, true, false, 4)
}  // namespace gemv
