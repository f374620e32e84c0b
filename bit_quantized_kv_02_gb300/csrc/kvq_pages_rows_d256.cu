// kvq_pages_rows_d256.cu — paged attention for few query rows, head_dim 256.
#include "kvq_pages_rows.cuh"

namespace kvq {
AttnKernel rows_kernel_d256(int fmt, int nm) { return rows_kernel_dim<256, false>(fmt, nm); }
}  // namespace kvq
