// kvq_pages_rows_d64.cu — paged attention for few query rows, head_dim 64.
#include "kvq_pages_rows.cuh"

namespace kvq {
AttnKernel rows_kernel_d64(int fmt, int nm) { return rows_kernel_dim<64>(fmt, nm); }
}  // namespace kvq
