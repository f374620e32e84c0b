// kvq_pages_attn.cu — launches of attention over the paged cache, and the
// kernel that joins what several CTAs computed of one item.
#include <algorithm>
#include <climits>

#include "kvq_internal.h"
#include "kvq_pages_attn.cuh"

namespace kvq {

namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinShare = 16;  // parts from which the warps of a block share a row

// Joins the parts of the items that start in CTA blockIdx.x and end in a later
// one.  Few parts: a warp per row.  Many (an item over a long context has
// hundreds, and their reads are what takes the time): the block's warps share a
// row's parts and sum up through shared memory.
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
  const bool share = h.parts > kJoinShare;
  const int step = share ? 1 : kJoinWarps;  // rows a block takes at once
  for (int r = blockIdx.y * step + (share ? 0 : warp); r < h.rows; r += gridDim.y * step) {
    // part i: slot 1 of the first CTA, slot 0 of the ones after it
    auto slot = [&](int i) { return (i ? first + 2 * i - 1 : first) * ROWS + r; };
    float M = -INFINITY;
    for (int i = lane; i < h.parts; i += 32) M = fmaxf(M, a.part_ml[2 * slot(i)]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float y[V] = {}, l = 0.0f;
#pragma unroll 4
    for (int i = share ? warp : 0; i < h.parts; i += share ? kJoinWarps : 1) {
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
    const int R = h.row0 + r;
    const long at = ((long)(h.q_row + R / a.rep) * a.q_heads + h.head * a.rep + R % a.rep) * D;
    if (!share) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
      for (int c = 0; c < V; c += 2) store_out2(a, at + lane * V + c, y[c] * inv, y[c + 1] * inv);
      continue;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) part[warp][lane * V + c] = y[c];
    if (lane == 0) part[warp][D] = l;
    __syncthreads();
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

template <int D>
const void* join_dim(int rows) {
  switch (rows) {
    case 8: return (const void*)pages_join_kernel<D, 8>;
    case 16: return (const void*)pages_join_kernel<D, 16>;
    case 24: return (const void*)pages_join_kernel<D, 24>;
    case 32: return (const void*)pages_join_kernel<D, 32>;
    case 128: return (const void*)pages_join_kernel<D, 128>;
    default: return (const void*)pages_join_kernel<D, 256>;
  }
}

size_t launch_smem(const AttnKernel& k, int batch) { return k.smem + (size_t)(batch + 1) * sizeof(long); }

// CTAs that an SM holds at once.
int resident(const kvq_pages* P, const AttnKernel& k, int batch) {
  const size_t each = launch_smem(k, batch) + k.static_smem + P->cta_smem + 127;
  return std::max(1, std::min(k.reg_ctas, (int)(P->sm_smem / each)));
}

// One attention launch and the join of what its CTAs shared; `rows`: query rows
// a CTA holds, `used`: the most that an item can have.
cudaError_t launch_kernel(const AttnKernel& k, AttnArgs a, int ctas, int rows, int used, cudaStream_t st) {
  void* args[] = {&a};
  cudaError_t e = launch_pdl(k.fn, dim3(ctas), dim3(k.threads), launch_smem(k, a.bv.batch) + (size_t)a.ring * k.unit, st, args);
  if (e != cudaSuccess) return e;
  const int D = a.pv.head_dim;
  const void* join = D == 64 ? join_dim<64>(rows) : D == 128 ? join_dim<128>(rows) : join_dim<256>(rows);
  const int y = std::max(1, std::min(std::min(rows, used), rows > 32 ? 32 : 4));
  return launch_pdl(join, dim3(ctas, y), dim3(kJoinWarps * 32), 0, st, args);
}

cudaError_t launch_rows(kvq_pages* P, AttnArgs a, bool masked, int max_rows, cudaStream_t st) {
  // As few row tiles of 8 as hold a sequence's rows, up to 32 rows (16 at head_dim
  // 256): the cache is then read once for all of them, and no product is made for
  // rows that are not there.  32 sequences of 4096 4-bit tokens, 8 / 16 / 24 / 32
  // rows, us: heads of 64 49 / 60 / 71 / 86, of 128 56 / 71 / 78 / 99, of 256
  // 37 / 44; 20 rows over 8-bit pages 60, in two turns of 16 rows 94.
  const int most = P->cfg.head_dim == 256 ? 16 : kRowsPerCta;
  const int blocks = (max_rows + most - 1) / most, nm = ((max_rows + blocks - 1) / blocks + 7) / 8;
  const AttnKernel& k = P->rows_fn[masked][nm - 1];
  a.min_units = 2;
  return launch_kernel(k, a, std::min(resident(P, k, a.bv.batch) * P->sm_count, kPagesCtas), 8 * nm, max_rows, st);
}

cudaError_t launch_tile(kvq_pages* P, AttnArgs a, bool masked, int max_rows, cudaStream_t st) {
  const AttnKernel& k = P->tile_fn[masked];
  a.min_units = 2;
  if (P->L.k_bits != 16) {
    const int left = P->max_smem - (int)(k.static_smem + launch_smem(k, a.bv.batch));
    a.ring = std::min(left / k.unit, kTileAhead);
    if (a.ring < 1) return cudaErrorInvalidConfiguration;  // (not reached: one of the largest units fits)
  }
  return launch_kernel(k, a, std::min(P->sm_count, kTileCtas), a.pv.head_dim == 256 ? kTileRows / 2 : kTileRows,
                       max_rows, st);
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
  for (int nm = 1; nm <= (D < 256 ? 4 : 2); ++nm) {
    P->rows_fn[0][nm - 1] = D == 64 ? rows_kernel_d64(fmt, nm) : D == 128 ? rows_kernel_d128(fmt, nm) : rows_kernel_d256(fmt, nm);
    P->rows_fn[1][nm - 1] = D == 64    ? rows_mask_kernel_d64(fmt, nm)
                            : D == 128 ? rows_mask_kernel_d128(fmt, nm)
                                       : rows_mask_kernel_d256(fmt, nm);
  }
  P->tile_fn[0] = D == 64 ? tile_kernel_d64(fmt) : D == 128 ? tile_kernel_d128(fmt) : tile_kernel_d256(fmt);
  P->tile_fn[1] = D == 64 ? tile_mask_kernel_d64(fmt) : D == 128 ? tile_mask_kernel_d128(fmt) : tile_mask_kernel_d256(fmt);
  cudaError_t e = cudaDeviceGetAttribute(&P->sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, P->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P->cta_smem, cudaDevAttrReservedSharedMemoryPerBlock, P->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P->max_smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, P->device);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < 10; ++i) {
    AttnKernel* k = i % 5 == 4 ? &P->tile_fn[i / 5] : &P->rows_fn[i / 5][i % 5];
    if (!k->fn) continue;
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, k->fn);
    if (e != cudaSuccess) return e;
    k->static_smem = at.sharedSizeBytes;
    e = cudaFuncSetAttribute(k->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, P->max_smem - (int)at.sharedSizeBytes);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k->reg_ctas, k->fn, k->threads, 0);
    if (e != cudaSuccess) return e;
    if (k->reg_ctas < 1) return cudaErrorInvalidConfiguration;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_attn(kvq_pages* P, AttnArgs& a, bool masked, int max_rows, bool rows_given, cudaStream_t st) {
  // Sequences with at most `few` rows (new tokens x query heads per kv head) go to
  // the few-rows kernel, the others to the many-rows one; a batch that may hold
  // both kinds launches both.  Over 16-bit pages that goes for a single sequence of
  // unknown rows too, since the kernel decides how its weights are rounded (where
  // they are given, the second launch would cost 10 us for nothing: 64 tokens at 4k,
  // 32 over 8 heads of 128, 39 us with one launch and 49 with two).  Measured, few /
  // many rows, us, 8 sequences of 8192 tokens, causal: 16-bit pages, 12 heads of 64: 32 rows
  // 52 / 61, 48 rows 97 / 61; 8 heads of 128: 59 / 62, 98 / 64; 2 heads of 256:
  // 48 / 52, 61 / 55.  4 bits, heads of 64: 48 rows 63 / 71, 64 rows 81 / 72, 128 rows 134 / 74;
  // heads of 128: 32 rows 55 / 61, 48 rows 69 / 62, 64 rows 88 / 63; heads of 256: 16 rows
  // 35 / 41, 32 rows 48 / 43, 48 rows 56 / 45.
  // So the causal limits over codes (128, 64 and 48 rows) stand above the crossing.  They are
  // where a many-rows kernel of 159, 99 and 61 us there crossed, and have been kept while it
  // became faster: both kernels round the weights alike over codes, but a lower limit would
  // change the order of sums of the calls between.
  // Masked: 16-bit pages, heads of 64: 32 rows 53 / 58, 48 rows 104 / 58; of 128: 60 / 63,
  // 99 / 65; of 256: 50 / 52, 64 / 53.  8 bits, heads of 64: 48 rows 71 / 72, 64 rows 90 / 73;
  // heads of 128: 32 rows 62 / 66, 48 rows 78 / 67; heads of 256: 16 rows 40 / 44, 32 rows
  // 53 / 47.  4 bits: 65 / 71, 82 / 71; 57 / 60, 69 / 61; 36 / 40, 49 / 42.
  const int D = P->cfg.head_dim;
  const int few = P->L.k_bits == 16 ? 32
                  : masked          ? (D == 64 ? 48 : (D == 128 ? 32 : 16))
                                    : (D == 64 ? 128 : (D == 128 ? 64 : 48));
  a.rows_lo = 0;
  a.rows_hi = INT_MAX;
  if (P->which == 1 || (P->which == 0 && max_rows <= few)) return launch_rows(P, a, masked, max_rows, st);
  if (P->which == 2 || (a.bv.batch == 1 && (rows_given || P->L.k_bits != 16))) return launch_tile(P, a, masked, max_rows, st);
  // Over codes the masked kernels take a batch that is known to be mixed in one launch (of
  // one without the hint all sequences may have few rows): the weights are
  // rounded alike by both, the few-rows kernel would be its largest form, and its launch
  // and join cost 10 us.  32 trees of 1 to 31 tokens over 500 to 8192 4-bit tokens, 32 over
  // 8 heads of 128: 205 us with both, 202 with one (187 with three dequantizing warps a
  // tensor).  The rule does not look at how many sequences have few rows, and loses where
  // most have: one launch / both, us, single tokens and trees of 64 over 4096 4-bit tokens,
  // 12 heads of 64, 32 over 8 of 128, 16 over 2 of 256: 63 and 1 242 / 138, 239 / 203, 111 /
  // 108; 32 and 32 244 / 206, 254 / 253, 240 / 248; 4 and 60 246 / 256, 261 / 281, 345 / 377;
  // 15 and 1 72 / 60, 78 / 89, 42 / 63; 8 and 8 73 / 70, 81 / 99, 78 / 100.
  if (masked && rows_given && P->L.k_bits != 16) return launch_tile(P, a, masked, max_rows, st);
  a.rows_lo = few;
  cudaError_t e = launch_tile(P, a, masked, max_rows, st);
  if (e != cudaSuccess) return e;
  a.rows_lo = 0;
  a.rows_hi = few;
  return launch_rows(P, a, masked, few, st);
}

}  // namespace kvq
