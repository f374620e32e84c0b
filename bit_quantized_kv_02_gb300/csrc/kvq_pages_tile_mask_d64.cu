// kvq_pages_tile_mask_d64.cu — paged attention with masks for many query rows, head_dim 64.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_mask_kernel_d64(int fmt) { return tile_kernel_dim<64, true>(fmt); }
}  // namespace kvq
