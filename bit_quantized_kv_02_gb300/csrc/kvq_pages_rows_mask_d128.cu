// kvq_pages_rows_mask_d128.cu — paged attention with masks for few query rows, head_dim 128.
#include "kvq_pages_rows.cuh"

namespace kvq {
AttnKernel rows_mask_kernel_d128(int fmt, int nm) { return rows_kernel_dim<128, true>(fmt, nm); }
}  // namespace kvq
