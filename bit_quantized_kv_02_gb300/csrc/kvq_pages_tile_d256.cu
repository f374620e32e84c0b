// kvq_pages_tile_d256.cu — paged attention for many query rows, head_dim 256.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_kernel_d256(int fmt) { return tile_kernel_dim<256>(fmt); }
}  // namespace kvq
