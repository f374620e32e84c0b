// kvq_pages_tile_mask_d128.cu — paged attention with masks for many query rows, head_dim 128.
#include "kvq_pages_tile.cuh"

namespace kvq {
AttnKernel tile_mask_kernel_d128(int fmt) { return tile_kernel_dim<128, true>(fmt); }
}  // namespace kvq
