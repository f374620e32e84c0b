// kvq_pages_rows_mask_d256.cu — paged attention with masks for few query rows, head_dim 256.
#include "kvq_pages_rows.cuh"

namespace kvq {
AttnKernel rows_mask_kernel_d256(int fmt, int nm) { return rows_kernel_dim<256, true>(fmt, nm); }
}  // namespace kvq
