// kvq_pages_tile_d128.cu — paged attention for many query rows, head_dim 128.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_kernel_d128(int fmt) { return tile_kernel_dim<128>(fmt); }
}  // namespace kvq
