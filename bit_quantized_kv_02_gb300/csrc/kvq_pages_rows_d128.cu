// kvq_pages_rows_d128.cu — paged attention for few query rows, head_dim 128.
#include "kvq_pages_rows.cuh"

namespace kvq {
AttnKernel rows_kernel_d128(int fmt, int nm) { return rows_kernel_dim<128, false>(fmt, nm); }
}  // namespace kvq
