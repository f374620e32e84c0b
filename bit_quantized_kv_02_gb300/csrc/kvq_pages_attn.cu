// kvq_pages_attn.cu — launches of attention over the paged cache, and the
// kernel that joins what several CTAs computed of one item.
#include <algorithm>
#include <climits>

#include "kvq_internal.h"
#include "kvq_pages_attn.cuh"

namespace kvq {

namespace {

constexpr int kJoinWarps = 8;

// Joins the parts of the items that start in CTA blockIdx.x and end in a later
// one.  A warp per share of the parts and all of a row's columns, then the warps'
// sums through shared memory: an item over a long context has hundreds of
// parts, and their reads are what takes the time.
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) pages_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int V = D / 32;  // columns of a lane
  __shared__ float part[kJoinWarps][D + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const SplitHead h = a.split[blockIdx.x];
  pdl_trigger();
  if (h.parts == 0) return;
  const long first = (long)blockIdx.x * 2 + 1;
  for (int r = blockIdx.y; r < h.rows; r += gridDim.y) {
    // part i: slot 1 of the first CTA, slot 0 of the ones after it
    auto slot = [&](int i) { return (i ? first + 2 * i - 1 : first) * ROWS + r; };
    float M = -INFINITY;
    for (int i = lane; i < h.parts; i += 32) M = fmaxf(M, a.part_ml[2 * slot(i)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float y[V] = {}, l = 0.0f;
#pragma unroll 4
    for (int i = warp; i < h.parts; i += kJoinWarps) {
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * slot(i));
      const float f = ml.x == -INFINITY ? 0.0f : fast_exp2(ml.x - M);
      l += f * ml.y;
      const float* src = a.part_o + slot(i) * D + lane * V;
#pragma unroll
      for (int c = 0; c < V; c += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + c);
        y[c] += f * x.x;
        y[c + 1] += f * x.y;
      }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) part[warp][lane * V + c] = y[c];
    if (lane == 0) part[warp][D] = l;
    __syncthreads();
    const int R = h.row0 + r;
    const long at = ((long)(h.q_row + R / a.rep) * a.q_heads + h.head * a.rep + R % a.rep) * D;
    for (int c = threadIdx.x * 2; c < D; c += kJoinWarps * 64) {
      float s0 = 0.0f, s1 = 0.0f, sl = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        s0 += part[w][c];
        s1 += part[w][c + 1];
        sl += part[w][D];
      }
      const float inv = sl > 0.0f ? 1.0f / sl : 0.0f;
      store_out2(a, at + c, s0 * inv, s1 * inv);
    }
    __syncthreads();
  }
}

const void* join_fn(int D, int rows) {
  if (D == 64) return rows == 16 ? (const void*)pages_join_kernel<64, 16> : (const void*)pages_join_kernel<64, 32>;
  if (D == 128) return rows == 16 ? (const void*)pages_join_kernel<128, 16> : (const void*)pages_join_kernel<128, 32>;
  return (const void*)pages_join_kernel<256, 16>;
}

cudaError_t launch_rows(kvq_pages* P, AttnArgs a, int max_rows, cudaStream_t st) {
  // Two row tiles per warp where a sequence may have more rows than one holds:
  // the cache is then read once for 32 rows.
  const int mt = max_rows > 16 && P->rows_fn[1].fn ? 2 : 1;
  const RowsKernel& k = P->rows_fn[mt - 1];
  const int ctas = std::min(k.ctas_per_sm * P->sm_count, kPagesCtas);
  a.min_units = 2;
  void* args[] = {&a};
  cudaError_t e = launch_pdl(k.fn, dim3(ctas), dim3(128), k.smem, st, args);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_fn(a.pv.head_dim, 16 * mt), dim3(ctas, std::min(std::max(max_rows, 1), 4)), dim3(kJoinWarps * 32), 0, st,
                    args);
}

}  // namespace

int pages_format(const kvq_pages* P) {
  const int k = P->L.k_bits, v = P->L.v_bits;
  if (k == 16) return P->cfg.dtype == KVQ_BF16 ? kFmtBf16 : kFmtF16;
  if (k == 8) return v == 8 ? kFmt88 : kFmt84;
  return v == 8 ? kFmt48 : kFmt44;
}

cudaError_t pages_attn_setup(kvq_pages* P) {
  const int D = P->cfg.head_dim, fmt = pages_format(P);
  for (int mt = 1; mt <= (D == 256 ? 1 : 2); ++mt) {
    RowsKernel k = D == 64 ? rows_kernel_d64(fmt, mt) : D == 128 ? rows_kernel_d128(fmt, mt) : rows_kernel_d256(fmt, mt);
    cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k.ctas_per_sm, k.fn, 128, k.smem);
    if (e != cudaSuccess) return e;
    if (k.ctas_per_sm < 1) return cudaErrorInvalidConfiguration;
    P->rows_fn[mt - 1] = k;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_attn(kvq_pages* P, AttnArgs& a, int max_rows, cudaStream_t st) {
  a.rows_lo = 0;
  a.rows_hi = INT_MAX;
  return launch_rows(P, a, max_rows, st);
}

}  // namespace kvq
