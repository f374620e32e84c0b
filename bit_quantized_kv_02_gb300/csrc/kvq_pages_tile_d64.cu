// kvq_pages_tile_d64.cu — paged attention for many query rows, head_dim 64.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_kernel_d64(int fmt) { return tile_kernel_dim<64>(fmt); }
}  // namespace kvq
