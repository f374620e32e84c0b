// kvq_pages.h — the paged cache: handle, page layout and internal launchers.
//
// Page layout.  A (page, kv head) is a run of 16-token records; a record holds
// the keys' rows, their metadata, the values' rows and their metadata, so one
// bulk copy brings a tile of both tensors and a page of any size is a whole
// number of records.
//  - 16-bit rows: columns in blocks of 64 (128 bytes), [block][16 tokens][128 B]
//    with 16-byte chunk j of token t stored at j ^ (t & 7).  That is the
//    128-byte-swizzled operand tile of the tensor cores (and free of bank
//    conflicts for ldmatrix), so a plain bulk copy puts it into shared memory
//    ready to use.
//  - 8-bit rows: head_dim codes in channel order.
//  - 4-bit rows: words of 8 channels, channel 2j at bits 4j, channel 2j+1 at
//    bits 16+4j: a shift and a mask by 0x000f000f give two neighbouring
//    channels in the two halves of a register.
//  - metadata: [16 tokens][head_dim / group] (zero, step) fp16 pairs.
#pragma once

#include <string>

#include "../../include/kvq.h"
#include "kvq_common.cuh"

namespace kvq {

constexpr int kPageTile = 16;      // tokens per record
constexpr int kPagesMaxBatch = 1024;
constexpr int kTreeWords = 4;      // most 64-bit words of a drafted token's mask
constexpr int kPagesCtas = 1024;   // most CTAs of an attention launch (partial slots are sized by it)
constexpr int kRowsPerCta = 32;    // most query rows a CTA of the few-rows kernel holds
constexpr int kTileCtas = 192;     // most CTAs of the many-rows kernel
constexpr int kTileRows = 256;     // most query rows a CTA of the many-rows kernel holds
constexpr int kTileAhead = 4;      // most units of codes that a warp of it copies ahead

struct PagesLayout {
  int k_bits, v_bits;
  int k_lg, v_lg;             // log2 of the channels per group
  int km_off, v_off, vm_off;  // byte offsets inside a record (keys' rows at 0)
  int tile_bytes;             // bytes of a record
};

// One layer of the pool as the kernels see it.
struct PagesView {
  char* base;
  PagesLayout L;
  int pages, heads, head_dim;
  int lg_pt;       // log2(page_tokens)
  int* err;        // bit 0: bad index, bit 1: a wait gave up, bit 2: no free pages, bit 3: negative length
};

__host__ __device__ inline long page_head_bytes(const PagesView& p) {
  return (long)(1 << (p.lg_pt - 4)) * p.L.tile_bytes;
}
// Record of token slot `slot` of (page, head).
__host__ __device__ inline char* record_of(const PagesView& p, int page, int head, int slot) {
  return p.base + ((long)page * p.heads + head) * page_head_bytes(p) + (long)(slot >> 4) * p.L.tile_bytes;
}

// Rows of one call (kvq_pages_batch), as the kernels see them.
struct BatchView {
  int batch, new_tokens;
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* table;
  long stride;
};

struct RopeView {
  const float* table;  // null: none
  int rows, dim, style;
  const int32_t* positions;
};

// How one item of attention work that several CTAs shared is put together:
// written by the CTA that holds the item's first part.
struct SplitHead {
  int parts;     // CTAs that hold a part; 0: nothing to join
  int rows;      // query rows of the item
  int row0;      // first query row inside the sequence
  int q_row;     // first new token of the sequence
  int head;      // kv head
  int pad[3];
};

struct AttnArgs {
  PagesView pv;
  BatchView bv;
  const void* q;
  void* out;
  long q_stride;
  float scale_log2;  // softmax scale * log2(e)
  int window, rep, q_heads;
  uint32_t rep_magic;  // ceil(2^16 / rep): n / rep == n * rep_magic >> 16 for n < 1024 and rep <= 64
  int q_bf16;        // type of q and out: 0 fp16, 1 bf16
  int q_aligned;     // rows of q may be read 16 bytes at a time
  int rows_lo, rows_hi;  // sequences with rows_lo < n * rep <= rows_hi are this launch's
  int ring;          // units that a warp copies ahead (many rows over codes; 0 otherwise)
  // the masked kernels: new tokens that a row sees (null: rows see every token of their sequence)
  const uint32_t* seen;
  int seen_words;    // 32-bit words a row
  const int32_t* positions;  // of the rows, for the window
  int min_units;     // fewest blocks of tokens worth a CTA of its own
  float* part_o;     // [CTA][2][rows][head_dim] partial sums of the first / last item of a CTA
  float* part_ml;    // [CTA][2][rows][2] their maxima and sums
  SplitHead* split;  // [CTA]
};

// An attention kernel: its dynamic shared memory (the batch's line of units comes
// on top), threads, the CTAs per SM that its registers allow, static shared memory,
// and what a unit copied ahead takes on top (many rows over codes).
struct AttnKernel {
  const void* fn;
  size_t smem;
  int threads;
  int reg_ctas;
  size_t static_smem;
  int unit;
};

}  // namespace kvq

struct kvq_pages {
  kvq_pages_config cfg;
  char* base = nullptr;
  kvq::PagesLayout L;
  size_t layer_bytes = 0;
  int* d_err = nullptr;
  float* d_part_o = nullptr;
  float* d_part_ml = nullptr;
  kvq::SplitHead* d_split = nullptr;
  int device = 0;
  int sm_count = 0;
  int sm_smem = 0, cta_smem = 0;  // shared memory of an SM, of it reserved per CTA
  int max_smem = 0;               // most that a CTA may have
  int which = 0;     // kernel choice (kvq_pages_set_kernel)
  // causal and masked kernels
  kvq::AttnKernel rows_fn[2][4] = {};  // few-rows kernel for 8, 16, 24 and 32 rows (8 and 16 at head_dim 256)
  kvq::AttnKernel tile_fn[2] = {};     // many-rows kernel
  int32_t* d_fresh = nullptr;  // kvq_pages_grow: [pages] free pages in the order they are dealt out
  void* d_keep = nullptr;      // kvq_pages_keep
  int32_t* d_copies = nullptr; // pairs of pages to copy: [0] their number, from [4] on sources, then targets
  std::string last_error;
};

namespace kvq {

PagesView pages_view(const kvq_pages* P, int layer);

cudaError_t launch_pages_append(const PagesView& pv, const BatchView& bv, const RopeView& rv, const void* k,
                                const void* v, int in_dtype, int page_bf16, long k_stride, long v_stride,
                                cudaStream_t st);
cudaError_t launch_pages_read(const PagesView& pv, const BatchView& bv, void* k_out, void* v_out, cudaStream_t st);
cudaError_t launch_norm_rope(const kvq_norm_rope_args& a, const RopeView& rv, cudaStream_t st);

// the few-rows kernel of each head_dim (one translation unit each) for a page
// format and number of row tiles of 8
enum { kFmtF16 = 0, kFmtBf16 = 1, kFmt88 = 2, kFmt44 = 3, kFmt84 = 4, kFmt48 = 5, kFormats = 6 };
int pages_format(const kvq_pages* P);
AttnKernel rows_kernel_d64(int fmt, int nm);
AttnKernel rows_kernel_d128(int fmt, int nm);
AttnKernel rows_kernel_d256(int fmt, int nm);
AttnKernel tile_kernel_d64(int fmt);
AttnKernel tile_kernel_d128(int fmt);
AttnKernel tile_kernel_d256(int fmt);
// the same with masks (trees, cross attention), in units of their own
AttnKernel rows_mask_kernel_d64(int fmt, int nm);
AttnKernel rows_mask_kernel_d128(int fmt, int nm);
AttnKernel rows_mask_kernel_d256(int fmt, int nm);
AttnKernel tile_mask_kernel_d64(int fmt);
AttnKernel tile_mask_kernel_d128(int fmt);
AttnKernel tile_mask_kernel_d256(int fmt);
cudaError_t launch_pages_attn(kvq_pages* P, AttnArgs& a, bool masked, int max_rows, bool rows_given, cudaStream_t st);
cudaError_t pages_attn_setup(kvq_pages* P);

// kvq_pages_branch.cu
cudaError_t launch_pages_tree(const PagesView& pv, const BatchView& bv, const int32_t* parents, int words, uint64_t* seen,
                              int32_t* positions, cudaStream_t st);
// (layers: how many from pv's on, `layer_bytes` apart)
cudaError_t launch_pages_keep(const PagesView& pv, int layers, long layer_bytes, const BatchView& bv, int max_new,
                              const uint8_t* keep, int32_t* lens_out, void* work, cudaStream_t st);
constexpr int kKeepSegs = 32768;  // segments of rows that its workspace has room for
size_t pages_keep_bytes();        // of the workspace
// `number`: device count of the pairs, of which there are at most `count`; null: count
cudaError_t launch_pages_copy(const PagesView& pv, int layers, long layer_bytes, const int32_t* src, const int32_t* dst,
                              int count, const int32_t* number, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesView& pv, const kvq_pages_fork_args& a, cudaStream_t st);
cudaError_t launch_pages_grow(const PagesView& pv, const kvq_pages_grow_args& a, int32_t* fresh, int32_t* copies,
                              cudaStream_t st);

}  // namespace kvq
