// kvq_pages_attn.cuh — what both attention kernels over the paged cache share:
// the division of the work, bulk copies with bounded waits, and the partial
// results of items that several CTAs hold.
//
// Work.  An item is a (sequence, kv head, block of query rows); its units are
// the blocks of tokens that its rows may see.  The units of all items stand in
// one line, sequence by sequence, and CTA c of C takes the units c*W/C ..
// (c+1)*W/C - 1: every CTA gets the same number, whatever the lengths are, and
// writes at most two partial results (the item it starts in and the item it
// ends in), so the workspace depends on the card and not on the lengths.  Where
// there are fewer items than CTAs (few-rows kernel) each item gets CTAs of its own
// instead, as many as its length asks for, if that leaves no CTA much more than
// its even share: no CTA then works on two items in turn.  Own CTAs / one line,
// us: 16 x 5 drafted tokens over 8-bit pages 68 / 76, 8 sequences of 8192 4-bit
// tokens 35 / 37, but 48 of 4096 98 / 75 and 64 of 1k to 32k 469 / 317.  All of it is worked out on the device from the lengths that hold when
// the kernel runs; a captured launch can be replayed with others.
#pragma once

#include <cuda_bf16.h>

#include "kvq_pages.h"

namespace kvq {

// ------------------------------------------------------------- primitives --

__device__ __forceinline__ void mbar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, int parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ unsigned long long time_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
constexpr unsigned long long kWaitNs = 2000000000ull;  // longest wait on a barrier
// Waits for the phase, by one thread.  False where `limit` ns pass first, which is
// recorded in *err and *dead (shared memory), or where another thread of the CTA has
// given up.  Short, and its loop not unrolled: a wait is written at many places of a
// kernel, and what a warp runs while it waits must not drive the others' code out of the
// instruction cache (64 polls between looks at the clock, which the compiler unrolled,
// made a kernel 240 KB long, and chunks over 8-bit pages 578 us against 484).
__device__ __forceinline__ bool cta_wait(uint32_t bar, int parity, int* dead, int* err,
                                         unsigned long long limit = kWaitNs) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = time_ns();
#pragma unroll 1
  do {
    if (mbar_try(bar, parity)) return true;
    if (*(volatile int*)dead) return false;
  } while (time_ns() - t0 < limit);
  *(volatile int*)dead = 1;
  atomicOr(err, 2);
  return false;
}
// The same by a warp, whose lanes decide together: each has its own clock, and the
// warp must not part.
__device__ __forceinline__ bool warp_wait(uint32_t bar, int parity, int* dead, int* err,
                                          unsigned long long limit = kWaitNs) {
  return __all_sync(0xffffffffu, cta_wait(bar, parity, dead, err, limit));
}
// After a wait that gave up, by a warp: the copies into the `n` stages from `stage`
// on (a ring of NS barriers at `bar`) that are still under way land, or `limit` ns
// pass.  `phase`: parity of stage `stage`; the ones behind the ring's end are a
// phase further.
template <int NS>
__device__ __forceinline__ void ring_drain(uint32_t bar, int stage, int phase, int n,
                                           unsigned long long limit = kWaitNs) {
  const unsigned long long t0 = time_ns();
  for (; n > 0; --n) {
    while (!mbar_try(bar + stage * 8, phase) && time_ns() - t0 < limit) {
    }
    if (++stage == NS) stage = 0, phase ^= 1;
  }
  __syncwarp();
}
// Bulk copy global -> shared; both addresses and the size multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, int bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// -------------------------------------------------------------------- work --

// A sequence of the call, clamped into the arrays: rows [s0, s0 + n), length
// len, first new token at position len - n.
struct Seq {
  int s0, n, len;
  int p0;  // len - n, may be negative
};

__device__ __forceinline__ Seq load_seq(const PagesView& pv, const BatchView& bv, int b, bool* bad) {
  const int a = bv.q_start[b], e = bv.q_start[b + 1], l = bv.lens[b];
  const long cap = bv.stride << pv.lg_pt;
  Seq s;
  s.s0 = min(max(a, 0), bv.new_tokens);
  s.n = min(max(e, s.s0), bv.new_tokens) - s.s0;
  s.len = (int)min((long)max(l, 0), min(cap, 1L << 30));
  *bad = a != s.s0 || e != s.s0 + s.n || l != s.len;
  s.p0 = s.len - s.n;
  return s;
}

// What is recorded of a sequence that load_seq calls bad.  A negative length, which growth
// leaves where pages ran out, has a bit of its own.
__device__ __forceinline__ int seq_error(const BatchView& bv, int b, const Seq& s) {
  return bv.lens[b] < 0 && bv.q_start[b] == s.s0 && bv.q_start[b + 1] == s.s0 + s.n ? 8 : 1;
}

// A sequence as attention takes it.  MASK: rows see the tokens before p0, and of
// those from p0 on the ones that a.seen names; without a.seen all tokens lie before p0.
template <bool MASK>
__device__ __forceinline__ Seq attn_seq(const AttnArgs& a, int b, bool* bad) {
  Seq s = load_seq(a.pv, a.bv, b, bad);
  if constexpr (MASK) {
    if (!a.seen) s.p0 = s.len;
    else if (s.n > 32 * a.seen_words) *bad = true;
  }
  return s;
}

// Which of the tokens c .. c + 31 a row of the call sees (masked kernels): bit i
// stands for token c + i.  A window hides none of the new tokens: it is no shorter
// than they are many.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs& a, const Seq& s, int row, int c) {
  const int o = c - s.p0, n = s.len - s.p0;  // place among the masked tokens, their number
  uint32_t v = o <= -32 ? 0xffffffffu : (o < 0 ? (1u << -o) - 1 : 0u);
  if (o > -32 && o < n) {
    const uint32_t* w = a.seen + (long)row * a.seen_words;
    const int i = o >> 5;  // -1 where the past ends among the 32
    const uint32_t lo = i >= 0 && i < a.seen_words ? w[i] : 0u, hi = i + 1 < a.seen_words ? w[i + 1] : 0u;
    uint32_t m = __funnelshift_r(lo, hi, o & 31);
    if (n - o < 32) m &= (1u << (n - o)) - 1;
    v |= m;
  }
  if (a.window > 0) {
    const int gone = max(min(a.positions[row], s.len - 1), s.p0) - a.window + 1 - c;
    if (gone > 0) v &= gone < 32 ? 0xffffffffu << gone : 0u;
  }
  return v;
}

// Tokens that rows [r0, r1) of the sequence may see, in blocks of BK: the
// first block and their number (at least one: an item without tokens still
// writes its zeros).
template <int BK, bool MASK>
__device__ __forceinline__ void row_blocks(const Seq& s, int rep, int window, int r0, int r1, int* lo, int* nb) {
  const int hi = MASK ? s.len : max(s.p0 + (r1 - 1) / rep + 1, 0);
  const int first = window > 0 ? max((long)s.p0 + (MASK ? 0 : r0 / rep) - window + 1, 0L) : 0;
  *lo = first / BK;
  *nb = max((hi + BK - 1) / BK - *lo, 1);
}

// One CTA's piece of an item.
struct Piece {
  int b, head;
  Seq s;
  int r0, rows;     // query rows [r0, r0 + rows) of the sequence (token * rep + head of the group)
  int blk, nblk;    // the piece: blocks [blk, blk + nblk)
  int has_first, has_last;  // the item's first / last block is in the piece
  int parts;                // pieces of the item, 0: by its units
  long item0, item1;        // the item's units
};

// The line of units, as one CTA sees it.  `pre` (shared memory behind the
// kernel's own, batch + 1 entries) holds the units before each sequence.
template <int BK, int ROWS>
struct Work {
  long* pre;
  long total;
  int ctas;
  int own;  // > 0: items have CTAs of their own, one per `own` blocks; pre counts CTAs
};

template <int BK, int ROWS, bool MASK>
__device__ __forceinline__ long seq_units(const AttnArgs& a, const Seq& s, int lane) {
  const int R = s.n * a.rep;
  if (R <= a.rows_lo || R > a.rows_hi) return 0;
  long sum = 0;
  for (int m = lane; m < (R + ROWS - 1) / ROWS; m += 32) {
    int lo, nb;
    row_blocks<BK, MASK>(s, a.rep, a.window, m * ROWS, min(R, (m + 1) * ROWS), &lo, &nb);
    sum += nb;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Units of a sequence's kv head, by one thread; *one: it has a single block of rows.
template <int BK, int ROWS, bool MASK>
__device__ __forceinline__ long seq_units_serial(const AttnArgs& a, const Seq& s, bool* one) {
  const int R = s.n * a.rep;
  *one = true;
  if (R <= a.rows_lo || R > a.rows_hi) return 0;
  *one = R <= ROWS;
  long sum = 0;
  for (int r0 = 0; r0 < R; r0 += ROWS) {
    int lo, nb;
    row_blocks<BK, MASK>(s, a.rep, a.window, r0, min(R, r0 + ROWS), &lo, &nb);
    sum += nb;
  }
  return sum;
}

// All threads of the CTA; leaves the line in *w, its units before each sequence
// in `pre`.  FEW: sequences have a block of rows or so, a thread each; else a warp
// each.
template <int BK, int ROWS, bool FEW, bool MASK>
__device__ __forceinline__ void plan_work(const AttnArgs& a, Work<BK, ROWS>* w, long* pre) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int alone = 1;
  if (FEW) {
    for (int b = threadIdx.x; b < a.bv.batch; b += blockDim.x) {
      bool bad, one;
      const Seq s = attn_seq<MASK>(a, b, &bad);
      pre[b + 1] = seq_units_serial<BK, ROWS, MASK>(a, s, &one);
      alone = alone && one;
      if (bad) atomicOr(a.pv.err, seq_error(a.bv, b, s));
    }
  } else {
    for (int b = warp; b < a.bv.batch; b += warps) {
      bool bad;
      const Seq s = attn_seq<MASK>(a, b, &bad);
      const long u = seq_units<BK, ROWS, MASK>(a, s, lane);
      if (lane == 0) {
        pre[b + 1] = u;
        if (bad) atomicOr(a.pv.err, seq_error(a.bv, b, s));
      }
    }
  }
  alone = __syncthreads_and(alone);
  if (warp == 0) {
    // sum over the sequences of f(units of a head), times the heads; stored as a running sum if `keep`
    auto over = [&](auto f, bool keep) {
      long run = 0;
      for (int b0 = 0; b0 < a.bv.batch; b0 += 32) {
        const int b = b0 + lane;
        long x = b < a.bv.batch ? f(pre[b + 1]) * a.pv.heads : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        x += run;
        if (keep && b < a.bv.batch) pre[b + 1] = x;
        run = __shfl_sync(0xffffffffu, x, 31);
      }
      return run;
    };
    long total, own = 0;
    if (FEW && alone && over([](long u) { return (long)(u > 0); }, false) <= gridDim.x) {
      total = over([](long u) { return u; }, false);
      own = max((total + gridDim.x - 1) / gridDim.x, (long)a.min_units);
      const long even = own;
      while (over([&](long u) { return (u + own - 1) / own; }, false) > gridDim.x) own += max(own / 8, 1L);
      if (own > even + even / 4 + 2) own = 0;
    }
    total = own ? over([&](long u) { return (u + own - 1) / own; }, true) : over([](long u) { return u; }, true);
    if (lane == 0) {
      pre[0] = 0;
      w->pre = pre;
      w->total = total;
      w->own = (int)own;
      w->ctas = own ? (int)total : (int)min((long)gridDim.x, (total + a.min_units - 1) / a.min_units);
    }
  }
  __syncthreads();
}

template <int BK, int ROWS>
__device__ __forceinline__ long cta_begin(const Work<BK, ROWS>* w, int c) {
  return w->total * c / w->ctas;
}
// The CTA whose range holds unit u.
template <int BK, int ROWS>
__device__ __forceinline__ int cta_of(const Work<BK, ROWS>* w, long u) {
  int c = (int)(((u + 1) * w->ctas - 1) / w->total);  // largest c with c*total/ctas <= u
  while (c > 0 && cta_begin(w, c) > u) --c;
  while (c + 1 < w->ctas && cta_begin(w, c + 1) <= u) ++c;
  return c;
}

// CTA cta's piece where items have CTAs of their own.
template <bool MASK, int BK, int ROWS>
__device__ __forceinline__ Piece own_piece(const AttnArgs& a, const Work<BK, ROWS>* w, int cta) {
  int lo = 0, hi = a.bv.batch;  // pre[lo] <= cta < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (w->pre[mid] <= cta) lo = mid;
    else hi = mid;
  }
  Piece p;
  p.b = lo;
  bool bad;
  p.s = attn_seq<MASK>(a, lo, &bad);
  const int per_head = (int)(w->pre[lo + 1] - w->pre[lo]) / a.pv.heads, at = cta - (int)w->pre[lo];
  p.head = at / per_head;
  const int part = at - p.head * per_head;
  int blk0, nb;
  p.r0 = 0;
  p.rows = p.s.n * a.rep;
  row_blocks<BK, MASK>(p.s, a.rep, a.window, 0, p.rows, &blk0, &nb);
  const int from = (int)((long)nb * part / per_head), to = (int)((long)nb * (part + 1) / per_head);
  p.blk = blk0 + from;
  p.nblk = to - from;
  p.has_first = part == 0;
  p.has_last = part == per_head - 1;
  p.parts = per_head;
  p.item0 = p.item1 = 0;
  return p;
}

// The piece that starts at unit u and ends by `end`; all lanes of a warp.
template <bool MASK, int BK, int ROWS>
__device__ __forceinline__ Piece find_piece(const AttnArgs& a, const Work<BK, ROWS>* w, long u, long end) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.bv.batch;  // pre[lo] <= u < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (w->pre[mid] <= u) lo = mid;
    else hi = mid;
  }
  Piece p;
  p.b = lo;
  bool bad;
  p.s = attn_seq<MASK>(a, lo, &bad);
  const long per_head = (w->pre[lo + 1] - w->pre[lo]) / a.pv.heads;
  p.head = (int)((u - w->pre[lo]) / per_head);
  const long base = w->pre[lo] + per_head * p.head;
  const long rel = u - base;
  const int R = p.s.n * a.rep, tiles = (R + ROWS - 1) / ROWS;
  long run = 0;
  int blk0 = 0, nb = 0, m = 0;
  for (int m0 = 0; m0 < tiles; m0 += 32) {
    int l = 0, n = 0;
    if (m0 + lane < tiles) row_blocks<BK, MASK>(p.s, a.rep, a.window, (m0 + lane) * ROWS, min(R, (m0 + lane + 1) * ROWS), &l, &n);
    long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + x > rel);
    if (hit) {
      const int src = __ffs(hit) - 1;
      nb = __shfl_sync(0xffffffffu, n, src);
      blk0 = __shfl_sync(0xffffffffu, l, src);
      run += __shfl_sync(0xffffffffu, x, src) - nb;
      m = m0 + src;
      break;
    }
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  p.r0 = m * ROWS;
  p.rows = min(R - p.r0, ROWS);
  p.item0 = base + run;
  p.item1 = p.item0 + nb;
  p.blk = blk0 + (int)(u - p.item0);
  p.nblk = (int)(min(end, p.item1) - u);
  p.has_first = u == p.item0;
  p.has_last = u + p.nblk == p.item1;
  p.parts = 0;
  return p;
}

__device__ __forceinline__ int page_index(const AttnArgs& a, int b, int tok) {
  return a.bv.table[b * a.bv.stride + (tok >> a.pv.lg_pt)];
}
// Records of one kv head: address of the one that holds token `tok` of a
// sequence, in the given page.  A page outside the pool is replaced by page 0
// and recorded.
struct PageRun {
  const char* base;
  long page_bytes;  // from a page to the next
  __device__ __forceinline__ PageRun(const PagesView& pv, int head)
      : base(pv.base + head * page_head_bytes(pv)), page_bytes(pv.heads * page_head_bytes(pv)) {}
  __device__ __forceinline__ const char* at(const AttnArgs& a, int page, int tok) const {
    if ((unsigned)page >= (unsigned)a.pv.pages) {
      atomicOr(a.pv.err, 1);
      page = 0;
    }
    return base + page * page_bytes + ((tok & ((1 << a.pv.lg_pt) - 1)) >> 4) * a.pv.L.tile_bytes;
  }
};

__device__ __forceinline__ void store_out2(const AttnArgs& a, long at, float x, float y) {
  if (a.q_bf16) static_cast<__nv_bfloat162*>(a.out)[at >> 1] = __floats2bfloat162_rn(x, y);
  else static_cast<__half2*>(a.out)[at >> 1] = __floats2half2_rn(x, y);
}

}  // namespace kvq
