// kvq_pages_branch.cu — sequences that branch, on the paged cache: masks of drafted
// trees, keeping some of a sequence's tokens, copying pages, and tables whose rows
// share pages (fork, grow).
//
// A tree's masks and a table's entries are a few KB: what these kernels cost is their
// launch and one chain of loads after another, so each keeps the chain short.  Moving
// tokens and copying pages are bound by memory.  Measured, each kernel alone with cold
// caches: masks of 16 trees of 64 tokens 6 us; fork of 64 rows of 250 pages 5 + 3 us (table,
// counts), of 256 rows of 1900 pages over a pool of 60000 6 + 4; growth of 64 rows by a
// token 12 us and 5 for the copies of shared last pages, of 256 rows by up to 600 tokens
// 24 + 4; 509 pages of 64 tokens, 40 heads of 128, 8- and 4-bit, four layers: 334 us, 6.5
// TB/s read and written (96 % of a copy).  Half of 8 sequences of 9k to 16k 4-bit tokens, 8 heads of 128, four layers at
// once: 6 + 138 us, 3.0 TB/s: a (head, token) is 144 bytes in four pieces, and a warp's
// access touches eleven lines of the L1 cache for four lines' worth of bytes.
#include <algorithm>

#include "kvq_internal.h"
#include "kvq_pages_attn.cuh"

namespace kvq {

namespace {

// The whole CTA of 1024 threads: exclusive prefix sums of one value a thread; *total: of all.
__device__ __forceinline__ int block_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  int v = sums[lane], s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += z;
  }
  const int base = __shfl_sync(0xffffffffu, s - v, warp);
  *total = __shfl_sync(0xffffffffu, s, 31);
  __syncthreads();
  return base + y - x;
}

// -------------------------------------------------------------------- tree --

constexpr int kTreeThreads = 64 * kTreeWords;  // a thread per drafted token

// A CTA per sequence.  A row's mask is its chain of parents, followed in shared
// memory (parents are smaller than their children, so a chain ends); its position is
// the chain's length behind the past.
__global__ void __launch_bounds__(kTreeThreads) pages_tree_kernel(PagesView pv, BatchView bv, const int32_t* parents,
                                                                 int words, uint64_t* seen, int32_t* positions) {
  __shared__ int up[kTreeThreads];
  const int b = blockIdx.x, i = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  bool bad;
  const Seq s = load_seq(pv, bv, b, &bad);
  if (bad || s.n > 64 * words) {  // (the same for all threads)
    if (i == 0) atomicOr(pv.err, seq_error(bv, b, s));
    return;
  }
  const long row = (long)s.s0 + i;
  if (i < s.n) {
    int p = parents[row];
    if (p < -1 || p >= i) {
      atomicOr(pv.err, 1);
      p = -1;
    }
    up[i] = p;
  }
  __syncthreads();
  if (i >= s.n) return;
  uint64_t m[kTreeWords] = {};
  int depth = 0;
  for (int j = i; j >= 0; j = up[j], ++depth) {
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
      if (j >> 6 == w) m[w] |= 1ull << (j & 63);
  }
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w)
    if (w < words) seen[row * words + w] = m[w];
  if (positions) positions[row] = s.p0 + depth - 1;
}

// -------------------------------------------------------------------- keep --

constexpr int kKeepThreads = 256;

// What a thread moves of every token of a (layer, head): 16 bytes of a row, or one
// (zero, step) pair.
struct Column {
  long at;        // of token 0 of a record, from the record's head
  int stride;     // from a token to the next
  int chunk, turn;  // 16-bit rows: chunk index inside the 128-byte row, 7 (its swizzle); else 0
  bool wide;        // 16 bytes, else 4
};

// Columns of one tensor's codes or values, and of its metadata.
__host__ __device__ __forceinline__ int row_columns(const PagesView& pv, int bits) { return pv.head_dim * bits / 128; }
__host__ __device__ __forceinline__ int meta_columns(const PagesView& pv, int bits, int lg) {
  return bits == 16 ? 0 : pv.head_dim >> lg;
}
__host__ __device__ __forceinline__ int columns(const PagesView& pv) {
  return row_columns(pv, pv.L.k_bits) + row_columns(pv, pv.L.v_bits) + meta_columns(pv, pv.L.k_bits, pv.L.k_lg) +
         meta_columns(pv, pv.L.v_bits, pv.L.v_lg);
}

__device__ __forceinline__ Column column_of(const PagesView& pv, int c) {
  const PagesLayout& L = pv.L;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int bits = side ? L.v_bits : L.k_bits, n = row_columns(pv, bits), off = side ? L.v_off : 0;
    if (c < n) {
      if (bits == 16) return {off + (c >> 3) * 2048, 128, c & 7, 7, true};
      return {off + c * 16, pv.head_dim * bits / 8, 0, 0, true};
    }
    c -= n;
  }
  const int n = meta_columns(pv, L.k_bits, L.k_lg);
  if (c < n) return {L.km_off + c * 4, n * 4, 0, 0, false};
  c -= n;
  return {L.vm_off + c * 4, meta_columns(pv, L.v_bits, L.v_lg) * 4, 0, 0, false};
}

// A token's place: its record's offset in a layer for head 0, and its number in the
// record in the low four bits (records are a multiple of 64 bytes).
__device__ __forceinline__ long place_of(const PagesView& pv, int page, int slot) {
  return (long)(record_of(pv, page, 0, slot) - pv.base) | (slot & 15);
}

// One column of all layers' heads, by its number: where its bytes lie for a token's place.
struct ColumnOf {
  Column col;
  char* base;
  __device__ __forceinline__ ColumnOf(const PagesView& pv, long layer_bytes, long unit) {
    const int ncol = columns(pv);
    const long lh = unit / ncol;  // layer * heads + head
    col = column_of(pv, (int)(unit - lh * ncol));
    base = pv.base + (lh / pv.heads) * layer_bytes + (lh % pv.heads) * page_head_bytes(pv) + col.at;
  }
  __device__ __forceinline__ char* at(long place) const {
    const int t = (int)(place & 15);
    return base + (place - t) + (t * col.stride + ((col.chunk ^ (t & col.turn)) << 4));
  }
  __device__ __forceinline__ void load(long place, uint4* x) const {
    if (col.wide) *x = *reinterpret_cast<const uint4*>(at(place));
    else x->x = *reinterpret_cast<const uint32_t*>(at(place));
  }
  __device__ __forceinline__ void store(long place, const uint4& x) const {
    if (col.wide) *reinterpret_cast<uint4*>(at(place)) = x;
    else *reinterpret_cast<uint32_t*>(at(place)) = x.x;
  }
};

// Places that token `from` of a sequence leaves and takes (`to`); {-1, -1}: it stays.
__device__ __forceinline__ long2 move_of(const PagesView& pv, const BatchView& bv, int b, int from, int to, bool report) {
  if (from == to) return make_long2(-1, -1);
  const int in = (1 << pv.lg_pt) - 1;
  const int pf = bv.table[b * bv.stride + (from >> pv.lg_pt)], pt = bv.table[b * bv.stride + (to >> pv.lg_pt)];
  if ((unsigned)pf >= (unsigned)pv.pages || (unsigned)pt >= (unsigned)pv.pages) {
    if (report) atomicOr(pv.err, 1);
    return make_long2(-1, -1);
  }
  return make_long2(place_of(pv, pf, from & in), place_of(pv, pt, to & in));
}

// Short sequences: the CTAs of row blockIdx.y go through one sequence's marks; each
// thread moves one column of one (layer, head) for all kept tokens.  No other thread
// touches those bytes, and tokens only move down, to places in their order: a thread
// that reads some tokens, then writes them, then goes on to the next never overwrites
// what it has yet to read.
__global__ void __launch_bounds__(kKeepThreads) pages_keep_kernel(PagesView pv, long layer_bytes, long units, BatchView bv,
                                                                 const uint8_t* keep, int32_t* lens_out) {
  __shared__ long2 move[kKeepThreads];
  __shared__ int sums[kKeepThreads / 32];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  bool bad;
  const Seq s = load_seq(pv, bv, b, &bad);
  if (bad) {
    if (blockIdx.x == 0 && tid == 0) {
      atomicOr(pv.err, seq_error(bv, b, s));
      if (lens_out) lens_out[b] = bv.lens[b];
    }
    return;
  }
  const long unit = (long)blockIdx.x * kKeepThreads + tid;
  const bool mine = unit < units;
  const ColumnOf col(pv, layer_bytes, mine ? unit : 0);
  const int skip = max(-s.p0, 0);  // rows that stand before the sequence
  int first = s.p0 + skip;         // where the next kept token goes
  for (int i0 = skip; i0 < s.n; i0 += kKeepThreads) {
    // the marks of 256 rows; places of the kept ones
    const int i = i0 + tid;
    const bool on = i < s.n && keep[(long)s.s0 + i] != 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, on);
    if (lane == 0) sums[warp] = __popc(ballot);
    __syncthreads();
    int before = __popc(ballot & ((1u << lane) - 1)), all = 0;
#pragma unroll
    for (int w = 0; w < kKeepThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (on) move[before] = move_of(pv, bv, b, s.p0 + i, first + before, blockIdx.x == 0);
    first += all;
    __syncthreads();
    if (mine) {
      constexpr int U = 8;  // tokens in flight
      for (int j = 0; j < all; j += U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u < all && move[j + u].x >= 0) col.load(move[j + u].x, &x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j + u < all && move[j + u].x >= 0) col.store(move[j + u].y, x[u]);
      }
    }
    __syncthreads();
  }
  if (lens_out && blockIdx.x == 0 && tid == 0) lens_out[b] = first;
}

// Long sequences: their rows in segments of 128, which many CTAs move at once.  A first
// kernel counts the kept rows before each segment.  Then a CTA takes a segment and 32
// columns, reads all of its kept tokens, says so, waits until the segments that its
// tokens go to have been read (they are never later ones, two at most), and writes.
// CTAs draw tickets in the order of the segments, so that of the steps that are not
// done the first waits for nobody: whoever holds it has nothing older to do, and what it
// writes to has been read.
constexpr int kSegRows = 128;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int load_acquire(const int* p) {
  int x;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];\n" : "=r"(x) : "l"(p) : "memory");
  return x;
}

struct KeepPlan {
  unsigned long long ticket;
  int segments;
};
// a segment: its sequence, its number there, kept rows before it, CTAs that have read it
struct KeepSeg {
  int b, at, before, done;
};

__device__ __forceinline__ int segments_of(const Seq& s) { return (s.n - max(-s.p0, 0) + kSegRows - 1) / kSegRows; }

__global__ void __launch_bounds__(kPlanThreads) pages_keep_plan_kernel(PagesView pv, BatchView bv, const uint8_t* keep,
                                                                      int32_t* lens_out, KeepPlan* plan, KeepSeg* seg) {
  __shared__ int sums[32];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  bool bad;
  const Seq s = load_seq(pv, bv, b, &bad);
  // segments of the sequences before this one
  int ahead = 0;
  if (tid < b) {
    bool skip;
    const Seq x = load_seq(pv, bv, tid, &skip);
    if (!skip) ahead = max(segments_of(x), 0);
  }
  int base;
  block_scan(ahead, sums, &base);
  const int rows = s.n - max(-s.p0, 0);
  const int segs = bad ? 0 : max(segments_of(s), 0);
  // Rows that several sequences name could make more segments than there is room for:
  // the line ends before the first sequence that does not fit.
  const bool full = base + segs > kKeepSegs;
  if (tid == 0) {
    if (b == 0) plan->ticket = 0;
    if (full ? base <= kKeepSegs : b == (int)gridDim.x - 1) plan->segments = full ? base : base + segs;
    if (bad || full) {
      atomicOr(pv.err, full ? 1 : seq_error(bv, b, s));
      if (lens_out) lens_out[b] = bv.lens[b];
    }
  }
  bad = bad || full;
  if (bad) return;
  const uint8_t* marks = keep + (long)s.s0 + (s.n - rows);
  constexpr int U = 4;  // segments in flight, a warp each
  for (int j0 = warp; j0 < segs; j0 += 32 * U) {
    unsigned hit[U][kSegRows / 32];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < kSegRows / 32; ++q) {
        const long i = (long)(j0 + 32 * u) * kSegRows + q * 32 + lane;
        hit[u][q] = __ballot_sync(0xffffffffu, i < rows && marks[i] != 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane == 0 && j0 + 32 * u < segs) {
        int n = 0;
#pragma unroll
        for (int q = 0; q < kSegRows / 32; ++q) n += __popc(hit[u][q]);
        seg[base + j0 + 32 * u] = {b, j0 + 32 * u, n, 0};
      }
  }
  __syncthreads();
  int run = 0;
  for (int j0 = 0; j0 < segs; j0 += kPlanThreads) {
    int all;
    const int j = j0 + tid, n = j < segs ? seg[base + j].before : 0;
    const int before = block_scan(n, sums, &all);
    if (j < segs) seg[base + j].before = run + before;
    run += all;
  }
  if (lens_out && tid == 0) lens_out[b] = max(s.p0, 0) + run;
}

// A step's chain of loads (ticket, segment, marks, page table, tokens) is spread over the
// steps before it: while a step's tokens come, the places of the next one's are found, the
// segment of the one after is read and the ticket of a third is drawn.  A step whose wait
// passes `limit` ns leaves its tokens where they are and is recorded.
__global__ void __launch_bounds__(kKeepThreads, 2) pages_keep_move_kernel(PagesView pv, long layer_bytes, long units,
                                                                         BatchView bv, const uint8_t* keep, KeepPlan* plan,
                                                                         KeepSeg* seg, unsigned long long limit) {
  constexpr int U = kSegRows / (kKeepThreads / 32);  // tokens of a warp
  __shared__ long2 move[2][kSegRows];
  __shared__ int sums[kSegRows / 32], ready;
  __shared__ uint32_t arrived[kKeepThreads];
  __shared__ long drawn[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const long blocks = (units + 31) / 32, total = plan->segments * blocks;
  struct Step {
    KeepSeg g;
    Seq s;
    int id, all;  // segment (-1: none), kept rows
    long unit;
  };
  // what a ticket stands for
  auto step_of = [&](long ticket) {
    Step st = {};
    st.id = -1;
    if (ticket >= total) return st;
    st.id = (int)(ticket / blocks);
    st.unit = (ticket - st.id * blocks) * 32 + lane;
    st.g = seg[st.id];
    bool bad;
    st.s = load_seq(pv, bv, st.g.b, &bad);
    return st;
  };
  // the places of its kept tokens
  auto find = [&](Step& st, long2* to) {
    if (st.id < 0) return;  // (all threads)
    const int skip = max(-st.s.p0, 0), first = st.s.p0 + skip, i = skip + st.g.at * kSegRows + tid;
    const bool on = tid < kSegRows && i < st.s.n && keep[(long)st.s.s0 + i] != 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, on);
    if (lane == 0 && warp < kSegRows / 32) sums[warp] = __popc(ballot);
    __syncthreads();
    int before = __popc(ballot & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kSegRows / 32; ++w) {
      if (w < warp) before += sums[w];
      st.all += sums[w];
    }
    if (tid >= st.all && tid < kSegRows) to[tid] = make_long2(-1, -1);
    if (on) to[before] = move_of(pv, bv, st.g.b, st.s.p0 + i, first + st.g.before + before, st.unit == lane);
  };
  if (tid == 0)
    for (int i = 0; i < 3; ++i) drawn[i] = (long)atomicAdd(&plan->ticket, 1ull);
  __syncthreads();
  Step now = step_of(drawn[0]), next = step_of(drawn[1]);
  long third = drawn[2];
  find(now, move[0]);
  for (int buf = 0; now.id >= 0; buf ^= 1) {
    __syncthreads();
    const bool mine = now.unit < units;
    const ColumnOf col(pv, layer_bytes, mine ? now.unit : 0);
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = u * (kKeepThreads / 32) + warp;
      x[u] = make_uint4(0, 0, 0, 0);
      const long from = move[buf][j].x;
      if (mine && from >= 0) col.load(from, &x[u]);
    }
    // while they come
    const KeepSeg& g = now.g;
    // segments that hold the rows which are written, [before, before + all) of the sequence's
    const int seg0 = g.before / kSegRows, seg1 = now.all > 0 ? min((g.before + now.all - 1) / kSegRows, g.at - 1) : -1;
    long fourth = 0;
    if (tid == 0) {
      fourth = (long)atomicAdd(&plan->ticket, 1ull);
      bool read = true;  // (mostly they have been read long ago)
      for (int k = seg0; k <= seg1; ++k) read = read && load_acquire(&seg[now.id - g.at + k].done) >= blocks;
      ready = read;
    }
    const Step after = step_of(third);
    find(next, move[buf ^ 1]);
    // every load has come back when its values can be stored
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) any |= x[u].x | x[u].y | x[u].z | x[u].w;
    *(volatile uint32_t*)&arrived[tid] = any;
    if (tid == 0) drawn[0] = fourth;
    __syncthreads();
    third = drawn[0];
    if (tid == 32) {  // (this step's tokens have been read)
      __threadfence();
      atomicAdd(&seg[now.id].done, 1);
    }
    const bool wait = !ready;
    __syncthreads();
    if (wait) {
      if (tid == 0) {
        const unsigned long long t0 = time_ns();
        bool late = false;
        for (int k = seg0; k <= seg1; ++k)
          while (!late && load_acquire(&seg[now.id - g.at + k].done) < blocks) late = time_ns() - t0 > limit;
        if (late) atomicOr(pv.err, 2);
        ready = !late;
      }
      __syncthreads();
    }
    if (ready) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = u * (kKeepThreads / 32) + warp;
        const long to = move[buf][j].y;
        if (mine && to >= 0) col.store(to, x[u]);
      }
    }
    now = next;
    next = after;
  }
}

// -------------------------------------------------------------------- copy --

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyBytes = kCopyThreads * kCopyUnroll * 16;  // of a page that a CTA moves at a time

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(PagesView pv, int layers, long layer_bytes,
                                                                 const int32_t* src, const int32_t* dst, int count,
                                                                 const int32_t* number) {
  pdl_wait();
  pdl_trigger();
  const int pairs = number ? min(*number, count) : count;
  const long bytes = pv.heads * page_head_bytes(pv), chunks = (bytes + kCopyBytes - 1) / kCopyBytes;
  for (long w = blockIdx.x; w < (long)pairs * layers * chunks; w += gridDim.x) {
    const long pl = w / chunks, chunk = w - pl * chunks;
    const int pair = (int)(pl / layers), layer = (int)(pl - (long)pair * layers);
    const int from = src[pair], to = dst[pair];
    if (from < 0 || to < 0) continue;
    if (from >= pv.pages || to >= pv.pages) {
      if (threadIdx.x == 0) atomicOr(pv.err, 1);
      continue;
    }
    const char* x = pv.base + layer * layer_bytes + from * bytes;
    char* y = pv.base + layer * layer_bytes + to * bytes;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const long at = chunk * kCopyBytes + (u * kCopyThreads + threadIdx.x) * 16;
      if (at < bytes) v[u] = *reinterpret_cast<const uint4*>(x + at);
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
      const long at = chunk * kCopyBytes + (u * kCopyThreads + threadIdx.x) * 16;
      if (at < bytes) *reinterpret_cast<uint4*>(y + at) = v[u];
    }
  }
}

// -------------------------------------------------------------------- fork --

constexpr int kForkThreads = 256;
constexpr int kForkEntries = 4;  // of a thread

// Row b of the new table from row parent[b] of the old one, kForkEntries entries a
// thread; the CTAs behind the table's copy reference counts.
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(PagesView pv, kvq_pages_fork_args a, int row_blocks) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / row_blocks;
  if (b >= a.rows_out) {
    const long i0 = (long)(blockIdx.x - a.rows_out * row_blocks) * (kForkThreads * kForkEntries) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kForkEntries; ++k) {
      const long i = i0 + k * kForkThreads;
      if (i < pv.pages) a.refs_out[i] = a.refs_in[i];
    }
    return;
  }
  const int p = a.parent[b];
  bool bad = p < -1 || p >= a.rows_in;
  int len = 0;
  long held = 0;  // pages that hold its tokens
  if (p >= 0 && !bad) {
    len = a.lens_in[p];
    const long tokens = len < 0 ? -1L - len : len;
    held = (tokens + (1 << pv.lg_pt) - 1) >> pv.lg_pt;
    bad = held > a.stride_in || held > a.stride_out;
  }
  if (bad) len = 0, held = 0;
  const long i0 = (long)(blockIdx.x - b * row_blocks) * (kForkThreads * kForkEntries) + threadIdx.x;
  int page[kForkEntries];
#pragma unroll
  for (int k = 0; k < kForkEntries; ++k) {
    const long i = i0 + k * kForkThreads;
    page[k] = i < held ? a.table_in[p * a.stride_in + i] : -1;
    if (i < held && (unsigned)page[k] >= (unsigned)pv.pages) bad = true, page[k] = -1;
  }
#pragma unroll
  for (int k = 0; k < kForkEntries; ++k)
    if (i0 + k * kForkThreads < a.stride_out) a.table_out[b * a.stride_out + i0 + k * kForkThreads] = page[k];
  if (bad) atomicOr(pv.err, 1);
  if (i0 == 0) a.lens_out[b] = len;
}

// References: one less for a name that left, one more for one that came.
__global__ void __launch_bounds__(kForkThreads) pages_refs_kernel(PagesView pv, kvq_pages_fork_args a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y;
  const long most = max(a.stride_in, a.stride_out), step = (long)gridDim.x * (kForkThreads * kForkEntries);
  for (long i0 = (long)blockIdx.x * (kForkThreads * kForkEntries) + threadIdx.x; i0 < most; i0 += step) {
    int was[kForkEntries], is[kForkEntries];
#pragma unroll
    for (int k = 0; k < kForkEntries; ++k) {
      const long i = i0 + k * kForkThreads;
      was[k] = b < a.rows_in && i < a.stride_in ? a.table_in[b * a.stride_in + i] : -1;
      is[k] = b < a.rows_out && i < a.stride_out ? a.table_out[b * a.stride_out + i] : -1;
    }
#pragma unroll
    for (int k = 0; k < kForkEntries; ++k) {
      if (was[k] == is[k]) continue;
      if (was[k] >= pv.pages) atomicOr(pv.err, 1);
      else if (was[k] >= 0) atomicSub(a.refs_out + was[k], 1);
      if (is[k] >= 0) atomicAdd(a.refs_out + is[k], 1);
    }
  }
}

// -------------------------------------------------------------------- grow --

constexpr int kGrowThreads = kPagesMaxBatch;  // a thread per sequence
constexpr int kGrowWarps = kGrowThreads / 32;
constexpr int kScan = 16;                     // reference counts that a thread has in flight

struct GrowArgs {
  kvq_pages_grow_args a;
  int32_t* fresh;   // [pages]
  int32_t *number, *src, *dst;
};

// One CTA deals out the pages: what a sequence gets depends on all before it.  A warp goes
// through a sequence's entries, once to count the fresh pages that they need and, where the
// sequence gets them, once to deal them out; one that does not get them, or that needs an
// entry outside the pool, has not been written to.  (Marks in the table, which the first
// look left for the second, were 1 to 2 us faster; all entries in one line, four a thread,
// 8 us slower.)
__global__ void __launch_bounds__(kGrowThreads) pages_grow_kernel(PagesView pv, GrowArgs g) {
  __shared__ int page[kGrowThreads];     // the page that holds the sequence's last tokens and is grown into, or -1
  __shared__ int first[kGrowThreads], last[kGrowThreads];  // entries of the table that the new tokens need
  __shared__ int need[kGrowThreads], from[kGrowThreads];   // fresh pages (then: does it get them?), and the first one's number
  __shared__ bool copies[kGrowThreads];
  __shared__ int sums[32], found_in[kScan * kGrowWarps];
  __shared__ int dealt;                  // fresh pages that are dealt out
  const kvq_pages_grow_args& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = a.sequences;
  pdl_wait();
  pdl_trigger();
  // ---- each sequence's part of the table
  const long cap = min(a.table_stride << pv.lg_pt, 1L << 30);
  int len = 0, n = 0, p = -1;
  bool bad = false;
  first[tid] = 0, last[tid] = -1;
  if (tid == 0) dealt = 0;
  if (tid < S) {
    len = a.lens[tid];
    const long count = (long)a.q_start[tid + 1] - a.q_start[tid];
    bad = len < 0 || count < 0 || len + count > cap;
    n = bad ? 0 : (int)count;
    if (n > 0) {
      const int f = len >> pv.lg_pt;
      if (len & ((1 << pv.lg_pt) - 1)) {
        p = a.table[tid * a.table_stride + f];
        if ((unsigned)p >= (unsigned)pv.pages) bad = true, n = 0, p = -1;
      }
      if (n > 0) first[tid] = f, last[tid] = (len + n - 1) >> pv.lg_pt;
    }
    if (bad && (len >= 0 || count < 0)) atomicOr(pv.err, 1);
  }
  page[tid] = p;
  __syncthreads();
  // entries that need a fresh page, but for the one that is grown into; -1: one lies outside the pool
  for (int b = warp; b < S; b += kGrowWarps) {
    int sum = 0;
    bool out = false;
    for (int i = first[b] + lane; i <= last[b]; i += 32) {
      const int old = a.table[b * a.table_stride + i];
      if (old >= pv.pages) out = true;
      else if (old < 0 || ((i != first[b] || page[b] < 0) && a.refs[old] > 1)) ++sum;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (__any_sync(0xffffffffu, out)) sum = -1;
    if (lane == 0) need[b] = sum;
  }
  __syncthreads();
  // (before the growers into a page are counted: a sequence that stays holds on to it)
  if (tid < S && need[tid] < 0) {
    atomicOr(pv.err, 1);
    bad = true, n = 0, p = -1;
    page[tid] = -1, last[tid] = first[tid] - 1, need[tid] = 0;
  }
  __syncthreads();
  bool copy = false;
  if (p >= 0) {
    const int r = a.refs[p];
    if (r > 1) {
      int before = 0;
      for (int c = 0; c < tid; ++c) before += page[c] == p;
      copy = before < r - 1;
    }
  }
  copies[tid] = copy;
  const int mine = tid < S ? need[tid] + copy : 0;
  int total;
  const int at = block_scan(mine, sums, &total);
  from[tid] = at;
  // ---- as many free pages as are wanted, the lowest first
  int found = 0;
  for (long p0 = 0; p0 < pv.pages && found < total; p0 += kScan * kGrowThreads) {
    unsigned hit[kScan];
#pragma unroll
    for (int k = 0; k < kScan; ++k) {
      const long i = p0 + k * kGrowThreads + tid;
      hit[k] = __ballot_sync(0xffffffffu, i < pv.pages && a.refs[i] == 0);
    }
#pragma unroll
    for (int k = 0; k < kScan; ++k)
      if (lane == 0) found_in[k * kGrowWarps + warp] = __popc(hit[k]);
    __syncthreads();
    int all;
    const int run = block_scan(tid < kScan * kGrowWarps ? found_in[tid] : 0, sums, &all);
    if (tid < kScan * kGrowWarps) found_in[tid] = run;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kScan; ++k)
      if (hit[k] >> lane & 1) {
        const int to = found + found_in[k * kGrowWarps + warp] + __popc(hit[k] & ((1u << lane) - 1));
        if (to < total) g.fresh[to] = (int)(p0 + k * kGrowThreads + tid);
      }
    found += all;
    __syncthreads();
  }
  // ---- who gets them: sequences in order, as far as the pages go
  const bool grows = n > 0, gets = grows && at + mine <= found;
  if (tid < S) a.lens_out[tid] = bad ? (len < 0 ? len : -1 - len) : gets ? len + n : grows ? -1 - len : len;
  if (grows && !gets) atomicOr(pv.err, 4);
  need[tid] = gets;
  if (gets) atomicMax(&dealt, at + mine);
  const int target = gets && copy ? g.fresh[at] : 0;  // (a copy is its sequence's first)
  int number;
  const int slot = block_scan(gets && copy, sums, &number);  // (its barriers publish the above)
  if (tid == 0) *g.number = number;
  if (gets && copy) g.src[slot] = p, g.dst[slot] = target;
  // An entry takes its fresh page and leaves there what it named: nobody's count may fall
  // before all have been looked at.  (The count of a page that was free is not above 1
  // before or after.)
  for (int b = warp; b < S; b += kGrowWarps) {
    if (!need[b]) continue;
    int run = from[b];
    for (int i0 = first[b]; i0 <= last[b]; i0 += 32) {
      const int i = i0 + lane;
      int32_t* e = a.table + b * a.table_stride + i;
      const bool in = i <= last[b];
      const int old = in ? *e : 0;
      const bool takes = in && (old < 0 || (i == first[b] && page[b] >= 0 ? copies[b] : a.refs[old] > 1));
      const unsigned hit = __ballot_sync(0xffffffffu, takes);
      if (takes) {
        const int k = run + __popc(hit & ((1u << lane) - 1)), f = g.fresh[k];
        *e = f;
        a.refs[f] = 1;
        g.fresh[k] = old;
      }
      run += __popc(hit);
    }
  }
  __syncthreads();
  for (int k = tid; k < dealt; k += kGrowThreads)
    if (g.fresh[k] >= 0) atomicSub(a.refs + g.fresh[k], 1);
}

int fork_blocks(long entries) { return (int)((entries + kForkThreads * kForkEntries - 1) / (kForkThreads * kForkEntries)); }

}  // namespace

cudaError_t launch_pages_tree(const PagesView& pv, const BatchView& bv, const int32_t* parents, int words, uint64_t* seen,
                              int32_t* positions, cudaStream_t st) {
  PagesView p = pv;
  BatchView b = bv;
  void* args[] = {&p, &b, &parents, &words, &seen, &positions};
  return launch_pdl((const void*)pages_tree_kernel, dim3(bv.batch), dim3(kTreeThreads), 0, st, args);
}

cudaError_t launch_pages_keep(const PagesView& pv, int layers, long layer_bytes, const BatchView& bv, int max_new,
                              const uint8_t* keep, int32_t* lens_out, void* work, cudaStream_t st) {
  PagesView p = pv;
  BatchView b = bv;
  long units = (long)layers * pv.heads * columns(pv);
  KeepPlan* plan = static_cast<KeepPlan*>(work);
  KeepSeg* seg = reinterpret_cast<KeepSeg*>(static_cast<char*>(work) + 256);
  if (max_new <= kKeepThreads || bv.new_tokens / kSegRows + bv.batch > kKeepSegs) {
    void* args[] = {&p, &layer_bytes, &units, &b, &keep, &lens_out};
    return launch_pdl((const void*)pages_keep_kernel, dim3((unsigned)((units + kKeepThreads - 1) / kKeepThreads), bv.batch),
                      dim3(kKeepThreads), 0, st, args);
  }
  void* args1[] = {&p, &b, &keep, &lens_out, &plan, &seg};
  cudaError_t e = launch_pdl((const void*)pages_keep_plan_kernel, dim3(bv.batch), dim3(kPlanThreads), 0, st, args1);
  if (e != cudaSuccess) return e;
  unsigned long long limit = kWaitNs;
  void* args2[] = {&p, &layer_bytes, &units, &b, &keep, &plan, &seg, &limit};
  const double most = (bv.new_tokens / kSegRows + bv.batch) * (double)((units + 31) / 32);
  return launch_pdl((const void*)pages_keep_move_kernel, dim3((unsigned)std::min(most, 152.0 * 2)), dim3(kKeepThreads), 0, st,
                    args2);
}

size_t pages_keep_bytes() { return 256 + sizeof(KeepSeg) * kKeepSegs; }

cudaError_t launch_pages_copy(const PagesView& pv, int layers, long layer_bytes, const int32_t* src, const int32_t* dst,
                              int count, const int32_t* number, cudaStream_t st) {
  PagesView p = pv;
  const long bytes = pv.heads * page_head_bytes(pv), chunks = (bytes + kCopyBytes - 1) / kCopyBytes;
  void* args[] = {&p, &layers, &layer_bytes, &src, &dst, &count, &number};
  const double work = (double)count * layers * chunks;
  return launch_pdl((const void*)pages_copy_kernel, dim3((unsigned)std::min(work, 152.0 * 8)), dim3(kCopyThreads), 0, st, args);
}

cudaError_t launch_pages_fork(const PagesView& pv, const kvq_pages_fork_args& x, cudaStream_t st) {
  PagesView p = pv;
  kvq_pages_fork_args a = x;
  int per = fork_blocks(a.stride_out);
  const int refs = a.refs_out != a.refs_in ? fork_blocks(pv.pages) : 0;
  void* args[] = {&p, &a, &per};
  cudaError_t e = launch_pdl((const void*)pages_fork_kernel, dim3((unsigned)(per * a.rows_out + refs)), dim3(kForkThreads), 0, st, args);
  if (e != cudaSuccess) return e;
  const long most = std::max(a.stride_in, a.stride_out);
  return launch_pdl((const void*)pages_refs_kernel,
                    dim3((unsigned)std::min((long)fork_blocks(most), 4096L), std::max(a.rows_in, a.rows_out)),
                    dim3(kForkThreads), 0, st, args);
}

cudaError_t launch_pages_grow(const PagesView& pv, const kvq_pages_grow_args& x, int32_t* fresh, int32_t* copies,
                              cudaStream_t st) {
  PagesView p = pv;
  GrowArgs g = {x, fresh, copies, copies + 4, copies + 4 + kPagesMaxBatch};
  void* args[] = {&p, &g};
  return launch_pdl((const void*)pages_grow_kernel, dim3(1), dim3(kGrowThreads), 0, st, args);
}

}  // namespace kvq
