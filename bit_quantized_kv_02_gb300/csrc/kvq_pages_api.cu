// kvq_pages_api.cu — the extern "C" boundary of the paged cache: validation,
// the pool's carve-up and dispatch.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>

#include "kvq_internal.h"
#include "kvq_pages.h"

using namespace kvq;

namespace {

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

kvq_status valid_page_tensor(const kvq_tensor_cfg& t, int D) {
  if (t.bits == 16) return KVQ_OK;
  if (t.bits < 2 || t.bits > 8) return KVQ_ERR_INVALID_ARG;
  if (t.axis != KVQ_PER_TOKEN && t.axis != KVQ_PER_CHANNEL) return KVQ_ERR_INVALID_ARG;
  if (t.mode != KVQ_ASYM && t.mode != KVQ_SYM) return KVQ_ERR_INVALID_ARG;
  if (t.group == 0 || (t.group < 0 && t.group != KVQ_WHOLE_VECTOR)) return KVQ_ERR_INVALID_ARG;
  if ((t.bits != 8 && t.bits != 4) || t.axis != KVQ_PER_TOKEN || t.mode != KVQ_ASYM) return KVQ_ERR_UNSUPPORTED;
  if (t.group != 32 && t.group != 64 && t.group != 128 && t.group != 256) return KVQ_ERR_UNSUPPORTED;
  return D % t.group == 0 ? KVQ_OK : KVQ_ERR_UNSUPPORTED;
}

kvq_status validate_pages(const kvq_pages_config* c) {
  if (!c) return KVQ_ERR_INVALID_ARG;
  if (c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->q_heads < 1) return KVQ_ERR_INVALID_ARG;
  if (c->page_tokens < 1 || c->q_heads % c->kv_heads) return KVQ_ERR_INVALID_ARG;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return KVQ_ERR_UNSUPPORTED;
  if (c->q_heads / c->kv_heads > 64 || c->kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  kvq_status s = valid_page_tensor(c->k, c->head_dim);
  if (s == KVQ_OK) s = valid_page_tensor(c->v, c->head_dim);
  if (s != KVQ_OK) return s;
  if ((c->k.bits == 16) != (c->v.bits == 16)) return KVQ_ERR_UNSUPPORTED;
  if (c->dtype != KVQ_F16 && c->dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (c->k.bits != 16 && c->dtype != KVQ_F16) return KVQ_ERR_INVALID_ARG;
  // the pool's bytes stay countable in 64 bits (a row is at most 512 bytes twice)
  const double rows = (double)c->layers * c->pages * c->page_tokens * c->kv_heads;
  return rows * 1024.0 < 9.0e15 ? KVQ_OK : KVQ_ERR_UNSUPPORTED;
}

PagesLayout pages_layout(const kvq_pages_config& c) {
  PagesLayout L = {};
  const int D = c.head_dim;
  L.k_bits = c.k.bits;
  L.v_bits = c.v.bits;
  L.k_lg = c.k.bits == 16 ? 0 : log2_of(c.k.group);
  L.v_lg = c.v.bits == 16 ? 0 : log2_of(c.v.group);
  L.km_off = 2 * D * c.k.bits;
  L.v_off = L.km_off + (c.k.bits == 16 ? 0 : kPageTile * (D >> L.k_lg) * 4);
  L.vm_off = L.v_off + 2 * D * c.v.bits;
  L.tile_bytes = L.vm_off + (c.v.bits == 16 ? 0 : kPageTile * (D >> L.v_lg) * 4);
  return L;
}

size_t layer_bytes_of(const kvq_pages_config& c, const PagesLayout& L) {
  return round256((size_t)c.pages * c.kv_heads * (c.page_tokens / kPageTile) * L.tile_bytes);
}

// partial results: floats of the outputs, rows of (maximum, sum)
void part_sizes(const kvq_pages_config& c, size_t* o, size_t* rows) {
  const size_t few = (size_t)kPagesCtas * 2 * (c.head_dim == 256 ? 16 : kRowsPerCta);
  const size_t many = (size_t)kTileCtas * 2 * (c.head_dim == 256 ? kTileRows / 2 : kTileRows);
  *rows = few > many ? few : many;
  *o = *rows * c.head_dim;
}

size_t carve_pages(const kvq_pages_config& c, kvq_pages* P) {
  const PagesLayout L = pages_layout(c);
  const size_t layer = layer_bytes_of(c, L);
  size_t o, rows;
  part_sizes(c, &o, &rows);
  size_t off = layer * c.layers;
  const size_t err = off;
  off += 256;
  const size_t split = off;
  off += round256(sizeof(SplitHead) * kPagesCtas);
  const size_t po = off;
  off += round256(o * 4);
  const size_t ml = off;
  off += round256(rows * 8);
  const size_t fresh = off;
  off += round256((size_t)c.pages * 4);
  const size_t copies = off;
  off += round256((4 + 2 * kPagesMaxBatch) * 4);
  const size_t keep = off;
  off += round256(pages_keep_bytes());
  if (P) {
    P->L = L;
    P->layer_bytes = layer;
    P->d_err = reinterpret_cast<int*>(P->base + err);
    P->d_split = reinterpret_cast<SplitHead*>(P->base + split);
    P->d_part_o = reinterpret_cast<float*>(P->base + po);
    P->d_part_ml = reinterpret_cast<float*>(P->base + ml);
    P->d_fresh = reinterpret_cast<int32_t*>(P->base + fresh);
    P->d_copies = reinterpret_cast<int32_t*>(P->base + copies);
    P->d_keep = P->base + keep;
  }
  return off;
}

kvq_status fail(kvq_pages* P, kvq_status s, const char* why) {
  try {
    P->last_error = why;
  } catch (...) {
  }
  return s;
}
kvq_status cuda_result(kvq_pages* P, cudaError_t e) {
  return e == cudaSuccess ? KVQ_OK : fail(P, KVQ_ERR_CUDA, cudaGetErrorString(e));
}

// Is p a multiple of its elements' size (a power of two)?
bool fits(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int element(int dtype) { return dtype == KVQ_F32 ? 4 : 2; }

// Do `rows` rows of `bytes` bytes, contiguous from `out` on, share a byte with as many
// rows `stride` bytes apart from `in` on?
bool overlap(const void* out, const void* in, int64_t rows, int64_t bytes, int64_t stride) {
  const int64_t o = (int64_t)reinterpret_cast<uintptr_t>(out), i = (int64_t)reinterpret_cast<uintptr_t>(in);
  // the first row of `in` that ends behind the start of `out`
  const int64_t r = o < i + bytes ? 0 : (o - i - bytes) / stride + 1;
  return r < rows && i + r * stride < o + rows * bytes;
}

// Do two arrays of so many bytes share one?
bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Does an array of so many bytes share one with those of the batch?
bool over_batch(const void* a, int64_t bytes, const BatchView& v) {
  return meet(a, bytes, v.q_start, 4 * (v.batch + 1L)) || meet(a, bytes, v.lens, 4L * v.batch) ||
         meet(a, bytes, v.table, 4L * v.batch * v.stride);
}

// Handle, layer and current device.
kvq_status usable(kvq_pages* P, int layer) {
  if (!P) return KVQ_ERR_INVALID_ARG;
  if (layer < 0 || layer >= P->cfg.layers) return fail(P, KVQ_ERR_INVALID_ARG, "layer out of range");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_result(P, e);
  return dev == P->device ? KVQ_OK : fail(P, KVQ_ERR_INVALID_ARG, "the current device is not the cache's");
}

kvq_status valid_batch(kvq_pages* P, const kvq_pages_batch* b, BatchView* v) {
  if (!b) return fail(P, KVQ_ERR_INVALID_ARG, "no batch");
  if (b->batch < 1 || b->batch > kPagesMaxBatch) return fail(P, KVQ_ERR_INVALID_ARG, "batch out of range");
  if (b->new_tokens < 0 || b->max_new < 0) return fail(P, KVQ_ERR_INVALID_ARG, "negative count of new tokens");
  if ((int64_t)b->new_tokens * P->cfg.q_heads > INT_MAX || (int64_t)b->new_tokens * P->cfg.kv_heads > INT_MAX)
    return fail(P, KVQ_ERR_UNSUPPORTED, "too many new tokens");
  if (!b->q_start || !b->lens || !b->table) return fail(P, KVQ_ERR_INVALID_ARG, "null batch array");
  if (!fits(b->q_start, 4) || !fits(b->lens, 4) || !fits(b->table, 4))
    return fail(P, KVQ_ERR_INVALID_ARG, "batch array not 4-byte aligned");
  if (b->table_stride < 1 || b->table_stride > (1L << 30)) return fail(P, KVQ_ERR_INVALID_ARG, "table stride out of range");
  *v = {b->batch, b->new_tokens, b->q_start, b->lens, b->table, (long)b->table_stride};
  return KVQ_OK;
}

// 0: usable, else the reason
const char* rope_fault(const kvq_rope* r, int D, bool positions, RopeView* v) {
  *v = {};
  if (!r) return nullptr;
  if (!r->table) return "null table of angles";
  if (reinterpret_cast<uintptr_t>(r->table) & 15) return "table of angles not 16-byte aligned";
  if (r->rows < 1) return "table of angles without rows";
  if (r->dim < 16 || r->dim > D || r->dim % 16) return "rotated channels out of range";
  if (r->style != KVQ_ROPE_PAIRS && r->style != KVQ_ROPE_HALVES) return "unknown rope style";
  if (positions && !r->positions) return "no positions";
  if (!fits(r->positions, 4)) return "positions not 4-byte aligned";
  *v = {r->table, r->rows, r->dim, r->style, r->positions};
  return nullptr;
}

}  // namespace

namespace kvq {
PagesView pages_view(const kvq_pages* P, int layer) {
  PagesView v = {};
  v.base = P->base + P->layer_bytes * layer;
  v.L = P->L;
  v.pages = P->cfg.pages;
  v.heads = P->cfg.kv_heads;
  v.head_dim = P->cfg.head_dim;
  v.lg_pt = log2_of(P->cfg.page_tokens);
  v.err = P->d_err;
  return v;
}
}  // namespace kvq

namespace {

// Attention of the rows of `batch`: causal, or masked, by `tree` or (null) over whole sequences.
kvq_status attend(kvq_pages_t P, int layer, const void* q, int q_dtype, int64_t q_stride, const kvq_pages_batch* batch,
                  bool masked, const kvq_tree* tree, float softmax_scale, int window, void* out, void* stream) {
  kvq_status s = usable(P, layer);
  if (s != KVQ_OK) return s;
  BatchView bv;
  s = valid_batch(P, batch, &bv);
  if (s != KVQ_OK) return s;
  const kvq_pages_config& c = P->cfg;
  if (q_dtype != KVQ_F16 && q_dtype != KVQ_BF16) return fail(P, KVQ_ERR_INVALID_ARG, "queries are fp16 or bf16");
  if (c.k.bits == 16 && q_dtype != c.dtype) return fail(P, KVQ_ERR_INVALID_ARG, "queries and 16-bit pages have one type");
  if (window < 0) return fail(P, KVQ_ERR_INVALID_ARG, "negative window");
  if (!(softmax_scale > 0.0f) && !std::isnan(softmax_scale)) softmax_scale = 1.0f / std::sqrt((float)c.head_dim);
  // in powers of two; not zero, which would turn a hidden score's -inf into NaN
  const float scale_log2 = std::max(softmax_scale * 1.44269504088896340736f, FLT_MIN);
  if (!std::isfinite(softmax_scale) || !std::isfinite(scale_log2))
    return fail(P, KVQ_ERR_INVALID_ARG, "softmax scale not finite");
  if (bv.new_tokens == 0) return KVQ_OK;
  if (!q || !out) return fail(P, KVQ_ERR_INVALID_ARG, "null queries or output");
  if (!fits(q, 2)) return fail(P, KVQ_ERR_INVALID_ARG, "queries not aligned to their type");
  if (q_stride < (int64_t)c.q_heads * c.head_dim) return fail(P, KVQ_ERR_INVALID_ARG, "stride shorter than a row");
  if (reinterpret_cast<uintptr_t>(out) & 15) return fail(P, KVQ_ERR_INVALID_ARG, "output not 16-byte aligned");
  if (overlap(out, q, bv.new_tokens, (int64_t)c.q_heads * c.head_dim * 2, q_stride * 2))
    return fail(P, KVQ_ERR_INVALID_ARG, "output and queries overlap");
  const int64_t out_bytes = (int64_t)bv.new_tokens * c.q_heads * c.head_dim * 2;
  if (over_batch(out, out_bytes, bv)) return fail(P, KVQ_ERR_INVALID_ARG, "output over the batch's arrays");
  if (tree && (meet(out, out_bytes, tree->seen, 8L * bv.new_tokens * tree->words) ||
               (tree->positions && meet(out, out_bytes, tree->positions, 4L * bv.new_tokens))))
    return fail(P, KVQ_ERR_INVALID_ARG, "output over the tree's arrays");
  AttnArgs a = {};
  a.pv = pages_view(P, layer);
  a.bv = bv;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.scale_log2 = scale_log2;
  a.window = window < (1 << 30) ? window : 0;  // (no sequence is longer)
  a.rep = c.q_heads / c.kv_heads;
  a.rep_magic = (65536 + a.rep - 1) / a.rep;
  a.q_heads = c.q_heads;
  a.q_bf16 = q_dtype == KVQ_BF16;
  a.q_aligned = (reinterpret_cast<uintptr_t>(q) & 15) == 0 && q_stride % 8 == 0;
  a.part_o = P->d_part_o;
  a.part_ml = P->d_part_ml;
  a.split = P->d_split;
  if (tree) {
    a.seen = reinterpret_cast<const uint32_t*>(tree->seen);
    a.seen_words = 2 * tree->words;
    a.positions = tree->positions;
  }
  const int max_new = batch->max_new > 0 && batch->max_new < bv.new_tokens ? batch->max_new : bv.new_tokens;
  return cuda_result(P, launch_pages_attn(P, a, masked, max_new * a.rep, batch->max_new > 0, static_cast<cudaStream_t>(stream)));
}

// A layer, or all of them: where they begin and how many they are.
kvq_status usable_layers(kvq_pages* P, int layer, PagesView* pv, int* layers) {
  const kvq_status s = usable(P, layer == KVQ_ALL_LAYERS ? 0 : layer);
  if (s != KVQ_OK) return s;
  *pv = pages_view(P, layer == KVQ_ALL_LAYERS ? 0 : layer);
  *layers = layer == KVQ_ALL_LAYERS ? P->cfg.layers : 1;
  return KVQ_OK;
}

// Do two arrays of 32-bit integers share one?
bool share(const int32_t* a, int64_t na, const int32_t* b, int64_t nb) { return meet(a, 4 * na, b, 4 * nb); }

}  // namespace

extern "C" {

kvq_status kvq_pages_bytes(const kvq_pages_config* c, kvq_bytes* out) {
  const kvq_status s = validate_pages(c);
  if (s != KVQ_OK) return s;
  if (!out) return KVQ_ERR_INVALID_ARG;
  const double rows = (double)c->layers * c->pages * c->page_tokens * c->kv_heads;
  std::memset(out, 0, sizeof(*out));
  out->packed = rows * c->head_dim * (c->k.bits + c->v.bits) / 8.0;
  if (c->k.bits != 16) out->metadata = rows * 4.0 * (c->head_dim / c->k.group + c->head_dim / c->v.group);
  size_t o, r;
  part_sizes(*c, &o, &r);
  out->workspace = 4.0 * (double)o + 8.0 * (double)r + 4.0 * c->pages + 4.0 * (4 + 2 * kPagesMaxBatch) +
                   (double)pages_keep_bytes();
  out->total = out->packed + out->metadata + out->workspace;
  out->elements = 2.0 * rows * c->head_dim;
  out->alloc = carve_pages(*c, nullptr);
  return KVQ_OK;
}

kvq_status kvq_pages_create(const kvq_pages_config* cfg, void* device_buf, size_t buf_bytes, void* stream,
                            kvq_pages_t* out) {
  const kvq_status s = validate_pages(cfg);
  if (s != KVQ_OK) return s;
  if (!device_buf || !out) return KVQ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(device_buf) & 255) return KVQ_ERR_INVALID_ARG;
  const size_t need = carve_pages(*cfg, nullptr);
  if (buf_bytes < need) return KVQ_ERR_BUFFER_TOO_SMALL;
  kvq_pages* P = new (std::nothrow) kvq_pages();
  if (!P) return KVQ_ERR_INVALID_ARG;
  P->cfg = *cfg;
  P->base = static_cast<char*>(device_buf);
  carve_pages(*cfg, P);
  cudaError_t e = cudaGetDevice(&P->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P->sm_count, cudaDevAttrMultiProcessorCount, P->device);
  if (e == cudaSuccess) e = pages_attn_setup(P);
  if (e == cudaSuccess) e = cudaMemsetAsync(device_buf, 0, need, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    delete P;
    return KVQ_ERR_CUDA;
  }
  *out = P;
  return KVQ_OK;
}

kvq_status kvq_pages_destroy(kvq_pages_t P) {
  if (!P) return KVQ_ERR_INVALID_ARG;
  delete P;
  return KVQ_OK;
}

kvq_status kvq_pages_append(kvq_pages_t P, int layer, const void* k, const void* v, int in_dtype, int64_t k_stride,
                            int64_t v_stride, const kvq_pages_batch* batch, const kvq_rope* rope, void* stream) {
  kvq_status s = usable(P, layer);
  if (s != KVQ_OK) return s;
  BatchView bv;
  s = valid_batch(P, batch, &bv);
  if (s != KVQ_OK) return s;
  RopeView rv;
  if (const char* why = rope_fault(rope, P->cfg.head_dim, false, &rv)) return fail(P, KVQ_ERR_INVALID_ARG, why);
  if (in_dtype != KVQ_F16 && in_dtype != KVQ_F32 && in_dtype != KVQ_BF16)
    return fail(P, KVQ_ERR_INVALID_ARG, "unknown dtype");
  if (bv.new_tokens == 0) return KVQ_OK;
  const int64_t row = (int64_t)P->cfg.kv_heads * P->cfg.head_dim;
  if (!k || !v) return fail(P, KVQ_ERR_INVALID_ARG, "null keys or values");
  if (!fits(k, element(in_dtype)) || !fits(v, element(in_dtype)))
    return fail(P, KVQ_ERR_INVALID_ARG, "keys or values not aligned to their type");
  if (k_stride < row || v_stride < row) return fail(P, KVQ_ERR_INVALID_ARG, "stride shorter than a row");
  return cuda_result(P, launch_pages_append(pages_view(P, layer), bv, rv, k, v, in_dtype, P->cfg.dtype == KVQ_BF16,
                                            k_stride, v_stride, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_read(kvq_pages_t P, int layer, const kvq_pages_batch* batch, void* k_out, void* v_out,
                          void* stream) {
  kvq_status s = usable(P, layer);
  if (s != KVQ_OK) return s;
  BatchView bv;
  s = valid_batch(P, batch, &bv);
  if (s != KVQ_OK) return s;
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15)
    return fail(P, KVQ_ERR_INVALID_ARG, "output not 16-byte aligned");
  if (bv.new_tokens == 0 || (!k_out && !v_out)) return KVQ_OK;
  return cuda_result(P, launch_pages_read(pages_view(P, layer), bv, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_attn(kvq_pages_t P, int layer, const void* q, int q_dtype, int64_t q_stride,
                          const kvq_pages_batch* batch, float softmax_scale, int window, void* out, void* stream) {
  return attend(P, layer, q, q_dtype, q_stride, batch, false, nullptr, softmax_scale, window, out, stream);
}

kvq_status kvq_pages_cross_attn(kvq_pages_t P, int layer, const void* q, int q_dtype, int64_t q_stride,
                                const kvq_pages_batch* batch, float softmax_scale, void* out, void* stream) {
  return attend(P, layer, q, q_dtype, q_stride, batch, true, nullptr, softmax_scale, 0, out, stream);
}

kvq_status kvq_pages_tree_attn(kvq_pages_t P, int layer, const void* q, int q_dtype, int64_t q_stride,
                               const kvq_pages_batch* batch, const kvq_tree* tree, float softmax_scale, int window,
                               void* out, void* stream) {
  if (!P) return KVQ_ERR_INVALID_ARG;
  if (!tree || !tree->seen) return fail(P, KVQ_ERR_INVALID_ARG, "no tree");
  if (tree->words < 1 || tree->words > kTreeWords) return fail(P, KVQ_ERR_INVALID_ARG, "words of a row out of range");
  if (!fits(tree->seen, 8) || !fits(tree->positions, 4))
    return fail(P, KVQ_ERR_INVALID_ARG, "tree not aligned to its types");
  if (window > 0 && window < 64 * tree->words)
    return fail(P, KVQ_ERR_UNSUPPORTED, "a window shorter than the tree's tokens");
  if (window > 0 && !tree->positions) return fail(P, KVQ_ERR_INVALID_ARG, "a window needs the tree's positions");
  return attend(P, layer, q, q_dtype, q_stride, batch, true, tree, softmax_scale, window, out, stream);
}

kvq_status kvq_pages_tree(kvq_pages_t P, const kvq_pages_batch* batch, const int32_t* parents, int words, uint64_t* seen,
                          int32_t* positions, void* stream) {
  kvq_status s = usable(P, 0);
  if (s != KVQ_OK) return s;
  BatchView bv;
  s = valid_batch(P, batch, &bv);
  if (s != KVQ_OK) return s;
  if (words < 1 || words > kTreeWords) return fail(P, KVQ_ERR_INVALID_ARG, "words of a row out of range");
  if (bv.new_tokens == 0) return KVQ_OK;
  if (!parents || !seen) return fail(P, KVQ_ERR_INVALID_ARG, "null parents or masks");
  if (!fits(parents, 4) || !fits(seen, 8) || !fits(positions, 4))
    return fail(P, KVQ_ERR_INVALID_ARG, "tree not aligned to its types");
  const int64_t ints = 4L * bv.new_tokens, masks = 8L * bv.new_tokens * words;
  if (meet(seen, masks, parents, ints) || over_batch(seen, masks, bv) ||
      (positions && (meet(positions, ints, parents, ints) || over_batch(positions, ints, bv) || meet(positions, ints, seen, masks))))
    return fail(P, KVQ_ERR_INVALID_ARG, "masks or positions over each other or over what is read");
  return cuda_result(P, launch_pages_tree(pages_view(P, 0), bv, parents, words, seen, positions,
                                          static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_keep(kvq_pages_t P, int layer, const kvq_pages_batch* batch, const uint8_t* keep, int32_t* lens_out,
                          void* stream) {
  PagesView pv;
  int layers;
  kvq_status s = usable_layers(P, layer, &pv, &layers);
  if (s != KVQ_OK) return s;
  BatchView bv;
  s = valid_batch(P, batch, &bv);
  if (s != KVQ_OK) return s;
  if (!keep && bv.new_tokens > 0) return fail(P, KVQ_ERR_INVALID_ARG, "null marks");
  if (!fits(lens_out, 4)) return fail(P, KVQ_ERR_INVALID_ARG, "lengths not 4-byte aligned");
  if (lens_out && over_batch(lens_out, 4L * bv.batch, bv))
    return fail(P, KVQ_ERR_INVALID_ARG, "new lengths over the batch's arrays");
  if (lens_out && meet(lens_out, 4L * bv.batch, keep, bv.new_tokens))
    return fail(P, KVQ_ERR_INVALID_ARG, "new lengths over the marks");
  if (bv.new_tokens == 0 && !lens_out) return KVQ_OK;
  const int max_new = batch->max_new > 0 && batch->max_new < bv.new_tokens ? batch->max_new : bv.new_tokens;
  return cuda_result(P, launch_pages_keep(pv, layers, (long)P->layer_bytes, bv, max_new, keep, lens_out, P->d_keep,
                                          static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_copy(kvq_pages_t P, int layer, const int32_t* src, const int32_t* dst, int count, void* stream) {
  PagesView pv;
  int layers;
  const kvq_status s = usable_layers(P, layer, &pv, &layers);
  if (s != KVQ_OK) return s;
  if (count < 0) return fail(P, KVQ_ERR_INVALID_ARG, "negative count of pages");
  if (count == 0) return KVQ_OK;
  if (!src || !dst) return fail(P, KVQ_ERR_INVALID_ARG, "null pages");
  if (!fits(src, 4) || !fits(dst, 4)) return fail(P, KVQ_ERR_INVALID_ARG, "pages not 4-byte aligned");
  return cuda_result(P, launch_pages_copy(pv, layers, (long)P->layer_bytes, src, dst, count, nullptr,
                                          static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_fork(kvq_pages_t P, const kvq_pages_fork_args* a, void* stream) {
  const kvq_status s = usable(P, 0);
  if (s != KVQ_OK) return s;
  if (!a) return fail(P, KVQ_ERR_INVALID_ARG, "no arguments");
  if (a->rows_in < 1 || a->rows_in > kPagesMaxBatch || a->rows_out < 1 || a->rows_out > kPagesMaxBatch)
    return fail(P, KVQ_ERR_INVALID_ARG, "rows out of range");
  if (a->stride_in < 1 || a->stride_in > (1L << 30) || a->stride_out < 1 || a->stride_out > (1L << 30))
    return fail(P, KVQ_ERR_INVALID_ARG, "table stride out of range");
  if (!a->parent || !a->table_in || !a->lens_in || !a->refs_in || !a->table_out || !a->lens_out || !a->refs_out)
    return fail(P, KVQ_ERR_INVALID_ARG, "null array");
  if (!fits(a->parent, 4) || !fits(a->table_in, 4) || !fits(a->lens_in, 4) || !fits(a->refs_in, 4) ||
      !fits(a->table_out, 4) || !fits(a->lens_out, 4) || !fits(a->refs_out, 4))
    return fail(P, KVQ_ERR_INVALID_ARG, "array not 4-byte aligned");
  const int64_t pages = P->cfg.pages;
  const struct {
    const int32_t* p;
    int64_t n;
  } in[] = {{a->parent, a->rows_out}, {a->table_in, a->rows_in * a->stride_in}, {a->lens_in, a->rows_in}, {a->refs_in, pages}},
    out[] = {{a->table_out, a->rows_out * a->stride_out}, {a->lens_out, a->rows_out}, {a->refs_out, pages}};
  for (int o = 0; o < 3; ++o) {
    for (const auto& i : in)
      if (share(out[o].p, out[o].n, i.p, i.n) && !(o == 2 && i.p == a->refs_in && a->refs_out == a->refs_in))
        return fail(P, KVQ_ERR_INVALID_ARG, "what is written lies over what is read");
    for (int x = 0; x < o; ++x)
      if (share(out[o].p, out[o].n, out[x].p, out[x].n)) return fail(P, KVQ_ERR_INVALID_ARG, "outputs overlap");
  }
  return cuda_result(P, launch_pages_fork(pages_view(P, 0), *a, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_pages_grow(kvq_pages_t P, const kvq_pages_grow_args* a, void* stream) {
  PagesView pv;
  int layers;
  const kvq_status s = usable_layers(P, KVQ_ALL_LAYERS, &pv, &layers);
  if (s != KVQ_OK) return s;
  if (!a) return fail(P, KVQ_ERR_INVALID_ARG, "no arguments");
  if (a->sequences < 1 || a->sequences > kPagesMaxBatch) return fail(P, KVQ_ERR_INVALID_ARG, "sequences out of range");
  if (a->table_stride < 1 || a->table_stride > (1L << 30)) return fail(P, KVQ_ERR_INVALID_ARG, "table stride out of range");
  if (!a->q_start || !a->lens || !a->table || !a->refs || !a->lens_out) return fail(P, KVQ_ERR_INVALID_ARG, "null array");
  if (!fits(a->q_start, 4) || !fits(a->lens, 4) || !fits(a->table, 4) || !fits(a->refs, 4) || !fits(a->lens_out, 4))
    return fail(P, KVQ_ERR_INVALID_ARG, "array not 4-byte aligned");
  const int64_t n = a->sequences, pages = P->cfg.pages, entries = n * a->table_stride;
  if (entries > INT_MAX) return fail(P, KVQ_ERR_UNSUPPORTED, "a table of more entries than 32 bits count");
  if ((a->lens_out != a->lens && share(a->lens_out, n, a->lens, n)) || share(a->lens_out, n, a->q_start, n + 1) ||
      share(a->lens_out, n, a->table, entries) || share(a->lens_out, n, a->refs, pages) ||
      share(a->table, entries, a->refs, pages) || share(a->table, entries, a->lens, n) ||
      share(a->table, entries, a->q_start, n + 1) || share(a->refs, pages, a->lens, n) ||
      share(a->refs, pages, a->q_start, n + 1))
    return fail(P, KVQ_ERR_INVALID_ARG, "arrays overlap");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pages_grow(pv, *a, P->d_fresh, P->d_copies, st);
  if (e == cudaSuccess)
    e = launch_pages_copy(pv, layers, (long)P->layer_bytes, P->d_copies + 4, P->d_copies + 4 + kPagesMaxBatch,
                          a->sequences, P->d_copies, st);
  return cuda_result(P, e);
}

kvq_status kvq_pages_set_kernel(kvq_pages_t P, int which) {
  if (!P || which < 0 || which > 2) return KVQ_ERR_INVALID_ARG;
  P->which = which;
  return KVQ_OK;
}

kvq_status kvq_pages_status(kvq_pages_t P, void* stream) {
  if (!P) return KVQ_ERR_INVALID_ARG;
  int word = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&word, P->d_err, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && word) e = cudaMemsetAsync(P->d_err, 0, sizeof(int), st);
  if (e != cudaSuccess) return cuda_result(P, e);
  if (!word) return KVQ_OK;
  // A wrong page shows nowhere else, so it goes before pages that ran out, which the
  // lengths tell; the lengths that those leave go behind.
  const kvq_status first = word & 2   ? KVQ_ERR_DEVICE_TIMEOUT
                           : word & 1 ? KVQ_ERR_BAD_INDEX
                           : word & 4 ? KVQ_ERR_OUT_OF_PAGES
                                      : KVQ_ERR_BAD_INDEX;
  const char* const index = word & 1   ? "a page, length or position was out of range"
                            : word & 4 ? nullptr
                                       : "a length was negative";
  char why[160] = "";
  for (const char* s : {word & 2 ? "a device-side wait gave up" : nullptr, index,
                        word & 4 ? "fewer free pages than the sequences needed" : nullptr})
    if (s) std::snprintf(why + std::strlen(why), sizeof(why) - std::strlen(why), "%s%s", *why ? "; " : "", s);
  return fail(P, first, why);
}

const char* kvq_pages_last_error(kvq_pages_t P) { return P ? P->last_error.c_str() : ""; }

kvq_status kvq_qk_norm_rope(const kvq_norm_rope_args* a, const kvq_rope* rope, void* stream) {
  if (!a || a->tokens < 0 || a->q_heads < 0 || a->kv_heads < 0) return KVQ_ERR_INVALID_ARG;
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
  if (a->dtype != KVQ_F16 && a->dtype != KVQ_F32 && a->dtype != KVQ_BF16) return KVQ_ERR_INVALID_ARG;
  if (a->norm && (!std::isfinite(a->eps) || a->eps < 0.0f)) return KVQ_ERR_INVALID_ARG;
  if (a->norm && (a->q_weight || a->k_weight) && a->weight_dtype != a->dtype && a->weight_dtype != KVQ_F32)
    return KVQ_ERR_INVALID_ARG;
  if (!fits(a->q, element(a->dtype)) || !fits(a->q_out, element(a->dtype)) || !fits(a->k, element(a->dtype)) ||
      !fits(a->k_out, element(a->dtype)))
    return KVQ_ERR_INVALID_ARG;
  if (a->norm && (!fits(a->q_weight, element(a->weight_dtype)) || !fits(a->k_weight, element(a->weight_dtype))))
    return KVQ_ERR_INVALID_ARG;
  RopeView rv;
  if (rope_fault(rope, a->head_dim, true, &rv)) return KVQ_ERR_INVALID_ARG;
  const int64_t qr = (int64_t)a->q_heads * a->head_dim, kr = (int64_t)a->kv_heads * a->head_dim;
  if (a->q_stride < qr || a->q_out_stride < qr || a->k_stride < kr || a->k_out_stride < kr) return KVQ_ERR_INVALID_ARG;
  if (a->tokens == 0 || (a->q_heads == 0 && a->kv_heads == 0)) return KVQ_OK;
  if ((int64_t)a->tokens * ((int64_t)a->q_heads + a->kv_heads) > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  if (a->q_heads && (!a->q || !a->q_out)) return KVQ_ERR_INVALID_ARG;
  if (a->kv_heads && (!a->k || !a->k_out)) return KVQ_ERR_INVALID_ARG;
  return launch_norm_rope(*a, rv, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
