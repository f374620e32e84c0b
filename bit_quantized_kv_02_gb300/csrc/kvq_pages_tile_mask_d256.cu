// kvq_pages_tile_mask_d256.cu — paged attention with masks for many query rows, head_dim 256.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_mask_kernel_d256(int fmt) { return tile_kernel_dim<256, true>(fmt); }
}  // namespace kvq
