// kvq_pages_write.cu — the row-wise kernels of the paged cache: norm of queries
// and keys with the rotary embedding, append of new tokens, and the read-back
// of what the pages hold.
//
// All three move rows of head_dim channels once through registers: a lane owns
// 8 neighbouring channels (16 bytes of a 16-bit row), head_dim / 8 lanes a row,
// and a warp one token at a time, so a token's angles are loaded once for all
// its heads and statistics (mean square, a group's minimum and maximum) are
// shuffles between a row's lanes.  For prompts they are bound by HBM bytes and,
// close behind, by issue slots: fp32 arithmetic goes two values an instruction
// (head norm of 65521 tokens 255 -> 226 us with the packed mean square and the
// approximate reciprocal root alone).  Prefetching the next token's rows, and
// blocks of a single batch of rows, were both slower (287 and 290 us).  Single
// tokens are bound by the launch and one chain of loads, so a token's heads
// spread over up to 8 warps.
// Measured: norm of 65521 tokens, 18 heads of 256, fp16, 225 us (5.4 TB/s read and
// written; a copy would take 180); append of 16 prompts of up to 4113 tokens, 40
// heads of 128, fp16 pages, 392 us with a read-back of the stored rows; 8 prompts
// of about 2000 tokens, 12 heads of 64, into 8- and 4-bit pages with the read-back
// 46 us (floor 18: the codes' arithmetic); 64 single tokens, in a graph: norm
// 3.7 us, append 6.6 us.
#include <cuda_bf16.h>

#include <algorithm>

#include "kvq_internal.h"
#include "kvq_pages_attn.cuh"
#include "kvq_pages_rows.cuh"  // (codes to values)

namespace kvq {

namespace {

constexpr int kThreads = 256;
constexpr int kRowWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 8 neighbouring elements as loaded: one or two 16-byte words, or element by
// element where the row is not 16-byte aligned.
template <typename T>
struct Row8 {
  uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Row8<T> load8(const T* p, bool aligned) {
  Row8<T> r;
  if (aligned) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i];
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Row8<T>& r, float* x) {
  const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f<T>(e[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x, bool aligned) {
  Row8<T> r;
  T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f<T>(x[i]);
  if (aligned) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = e[i];
  }
}

// A lane's angles: its 8 channels' cosines and signed sines, the lane that
// holds the partners (pairs (i, i + dim/2)), and whether the channels turn.
struct Turn {
  float c[8], s[8];
  int partner;
  bool on, halves;
};

__device__ __forceinline__ Turn load_turn(const RopeView& rv, long row, int c0, int lane) {
  Turn t;
  t.halves = rv.style == KVQ_ROPE_HALVES;
  t.on = rv.table != nullptr && c0 < rv.dim;
  t.partner = lane;
  if (!t.on) return t;
  const float* tab = rv.table + row * rv.dim;
  if (!t.halves) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(tab + c0));
    const float4 b = __ldg(reinterpret_cast<const float4*>(tab + c0) + 1);
    const float cs[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[2 * i] = t.c[2 * i + 1] = cs[2 * i];
      t.s[2 * i] = -cs[2 * i + 1];
      t.s[2 * i + 1] = cs[2 * i + 1];
    }
  } else {
    const int half = rv.dim / 2;
    const bool hi = c0 >= half;
    t.partner = lane + (hi ? -half / 8 : half / 8);
    const float* q = tab + 2 * (hi ? c0 - half : c0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(q) + i);
      t.c[2 * i] = a.x;
      t.s[2 * i] = hi ? a.y : -a.y;
      t.c[2 * i + 1] = a.z;
      t.s[2 * i + 1] = hi ? a.w : -a.w;
    }
  }
  return t;
}

// (a c - b s, b c + a s), each product and sum rounded once (the same numbers
// whatever the compiler fuses elsewhere: quantized pages round from them).
// Every lane of the warp calls it.
__device__ __forceinline__ void turn8(const Turn& t, float* x) {
  float p[8];
  if (t.halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], t.partner);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
  }
  if (t.on) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // (the sums one by one: a packed one may be fused with the products)
      const float2 y = mul2(make_float2(x[i], x[i + 1]), make_float2(t.c[i], t.c[i + 1]));
      const float2 z = mul2(make_float2(p[i], p[i + 1]), make_float2(t.s[i], t.s[i + 1]));
      x[i] = __fadd_rn(y.x, z.x), x[i + 1] = __fadd_rn(y.y, z.y);
    }
  }
}

// ------------------------------------------------------------- norm + rope --

struct NormArgs {
  const void *q, *k;
  void *q_out, *k_out;
  long qs, ks, qos, kos;
  const void *qw, *kw;
  int tokens, q_heads, kv_heads, norm, w_f32;
  float eps;
  int lg_wpt;       // log2 of the warps that share a token
  int aligned;      // every row may be moved 16 bytes at a time
  int w_aligned;    // the weights too
};

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, bool aligned, int c0, float* x) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.0f;
  } else if (w_f32) {
    unpack8(load8(static_cast<const float*>(w) + c0, aligned), x);
  } else {
    unpack8(load8(static_cast<const T*>(w) + c0, aligned), x);
  }
}

template <typename T, int D, int U>
__device__ __forceinline__ void norm_rows(const T* src, T* dst, int heads, int sub, int nsub, int lane, bool norm,
                                          float eps, const float* w, const Turn& turn, bool bad, bool aligned) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int rg = lane / LPR, c0 = (lane % LPR) * 8;
  // U rows in flight per lane
  for (int h0 = sub * RPW; h0 < heads; h0 += nsub * RPW * U) {
    Row8<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = min(h0 + u * nsub * RPW + rg, heads - 1);
      r[u] = load8(src + (long)h * D + c0, aligned);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hu = h0 + u * nsub * RPW;
      if (hu >= heads) break;
      float x[8];
      unpack8(r[u], x);
      if (norm) {
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) s2 = fma2(make_float2(x[i], x[i + 1]), make_float2(x[i], x[i + 1]), s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 y = mul2(mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv)), make_float2(w[i], w[i + 1]));
          x[i] = y.x, x[i + 1] = y.y;
        }
      }
      turn8(turn, x);
      if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __int_as_float(0x7fffffff);
      }
      const int h = hu + rg;
      if (h < heads) store8(dst + (long)h * D + c0, x, aligned);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(NormArgs a, RopeView rv) {
  constexpr int LPR = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nsub = 1 << a.lg_wpt, sub = warp & (nsub - 1);
  const int c0 = (lane % LPR) * 8;
  pdl_wait();
  pdl_trigger();
  float qw[8], kw[8];
  if (a.norm) {
    load_weight<T>(a.q_heads ? a.qw : nullptr, a.w_f32, a.w_aligned, c0, qw);
    load_weight<T>(a.kv_heads ? a.kw : nullptr, a.w_f32, a.w_aligned, c0, kw);
  }
  const long step = (long)gridDim.x * (kRowWarps >> a.lg_wpt);
  for (long t = (long)blockIdx.x * (kRowWarps >> a.lg_wpt) + (warp >> a.lg_wpt); t < a.tokens; t += step) {
    const int row = rv.table ? rv.positions[t] : 0;
    const bool bad = rv.table && (row < 0 || row >= rv.rows);
    const Turn turn = load_turn(rv, bad ? 0 : row, c0, lane);
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    if (a.q_heads)
      norm_rows<T, D, U>(static_cast<const T*>(a.q) + t * a.qs, static_cast<T*>(a.q_out) + t * a.qos, a.q_heads, sub, nsub,
                         lane, a.norm, a.eps, qw, turn, bad, a.aligned);
    if (a.kv_heads)
      norm_rows<T, D, 2>(static_cast<const T*>(a.k) + t * a.ks, static_cast<T*>(a.k_out) + t * a.kos, a.kv_heads, sub,
                         nsub, lane, a.norm, a.eps, kw, turn, bad, a.aligned);
  }
}

// Warps per token: as many blocks as two waves of the card need, one warp a
// token beyond.
int lg_warps_per_token(long tokens, long rows_per_warp_pass) {
  int lg = 0;
  while (lg < 3 && (tokens << lg) < 2L * 152 * kRowWarps && (1L << lg) < rows_per_warp_pass) ++lg;
  return lg;
}

template <typename T>
cudaError_t launch_norm_t(const kvq_norm_rope_args& x, const RopeView& rv, NormArgs a, cudaStream_t st) {
  const int rpw = 32 / (x.head_dim / 8);
  a.lg_wpt = lg_warps_per_token(x.tokens, (x.q_heads + x.kv_heads + rpw - 1) / rpw);
  const long per = kRowWarps >> a.lg_wpt;
  const long blocks = std::min((x.tokens + per - 1) / per, 152L * 8 * 4);
  const void* fn = x.head_dim == 64    ? (const void*)norm_rope_kernel<T, 64>
                   : x.head_dim == 128 ? (const void*)norm_rope_kernel<T, 128>
                                       : (const void*)norm_rope_kernel<T, 256>;
  RopeView r = rv;
  void* args[] = {&a, &r};
  return launch_pdl(fn, dim3((unsigned)blocks), dim3(kThreads), 0, st, args);
}

// ------------------------------------------------------------------ append --

// Where a new-token row of the call goes: page, slot and angle row, or page -1.
struct Place {
  int page, slot, turn;
};

// Places of `count` rows from t0 (no more than threads), by the whole block: every
// sequence's bounds and length are read at once, each row learns its sequence, and a
// thread a row follows the table, so a row costs two dependent loads whatever the batch
// and the count are.  A sequence whose length or rows do not fit has no places.  Only then
// can two sequences name the same row: the rows look for theirs one by one, and the first
// sequence that fits has it.
__device__ __forceinline__ void find_places(const PagesView& pv, const BatchView& bv, const RopeView* rv, long t0,
                                            int count, Place* place) {
  if (threadIdx.x < count) place[threadIdx.x] = {-1, -1, 0};  // (slot: the row's sequence, until it has a place)
  __syncthreads();
  int misfit = 0;
  for (int b = threadIdx.x; b < bv.batch; b += kThreads) {
    bool bad;
    const Seq s = load_seq(pv, bv, b, &bad);
    if (bad) {  // its clamped rows would stand at other positions: none is touched
      if (t0 == 0) atomicOr(pv.err, seq_error(bv, b, s));  // (one block reports)
      misfit = 1;
      continue;
    }
    const long lo = max(t0, (long)s.s0), hi = min(t0 + count, (long)s.s0 + s.n);
    for (long t = lo; t < hi; ++t) place[t - t0].slot = b;
  }
  misfit = __syncthreads_or(misfit);
  if (threadIdx.x < count) {
    const long t = t0 + threadIdx.x;
    int b = place[threadIdx.x].slot;
    bool bad = false;
    Seq s = {};
    if (misfit) {
      for (b = 0; b < bv.batch; ++b) {
        s = load_seq(pv, bv, b, &bad);
        if (!bad && t >= s.s0 && t < (long)s.s0 + s.n) break;
      }
      if (b == bv.batch) b = -1;
    } else if (b >= 0) {
      s = load_seq(pv, bv, b, &bad);
    }
    Place p = {-1, 0, 0};
    const long pos = s.p0 + (t - s.s0);
    if (b >= 0 && pos >= 0) {
      const int page = bv.table[b * bv.stride + (pos >> pv.lg_pt)];
      bool ok = (unsigned)page < (unsigned)pv.pages;
      long turn = 0;
      if (rv && rv->table) {
        turn = rv->positions ? rv->positions[t] : pos;
        ok = ok && turn >= 0 && turn < rv->rows;
      }
      if (ok) p = {page, (int)(pos & ((1 << pv.lg_pt) - 1)), (int)turn};
      else atomicOr(pv.err, 1);
    }
    place[threadIdx.x] = p;
  }
  __syncthreads();
}

// One row's 8 channels from c0 on into its record (`rec` + `off`): 16-bit, or
// codes with the group's metadata.  Every lane of the warp calls it.
template <int D, bool QUANT>
__device__ __forceinline__ void put8(char* rec, int off, int meta_off, int bits, int lg_group, int slot, int c0,
                                     const float* x, int page_bf16, bool write) {
  const int t = slot & 15;
  if (!QUANT) {
    if (!write) return;
    char* dst = rec + off + (c0 >> 6) * 2048 + t * 128 + ((((c0 >> 3) & 7) ^ (t & 7)) << 4);
    if (page_bf16) store8(reinterpret_cast<__nv_bfloat16*>(dst), x, true);
    else store8(reinterpret_cast<__half*>(dst), x, true);
    return;
  }
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
  for (int o = 1; o < (1 << (lg_group - 3)); o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  float z, s;
  group_params(mn, mx, 0.0f, bits, 0, 0, &z, &s);
  if (!write) return;
  const float r = s == 0.0f ? 0.0f : __frcp_rn(s);
  uint32_t q[8];
  // quant_code_fast's codes, two values an instruction: rounded by adding and
  // removing 1.5 * 2^23, and taken again one by one where a quotient is near a
  // half-integer.  z <= x <= z + (2^bits - 1) s keeps them in range unclamped.
  bool sure = r >= 0x1p-125f || s == 0.0f;
  const float2 big = make_float2(12582912.0f, 12582912.0f), small = make_float2(-12582912.0f, -12582912.0f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 num = add2(make_float2(x[i], x[i + 1]), make_float2(-z, -z));
    const float2 q0 = make_float2(__fmul_rn(num.x, r), __fmul_rn(num.y, r));
    const float2 m = add2(q0, big);
    const float2 c = add2(m, small);
    sure = sure && fabsf(__fsub_rn(q0.x, c.x)) < 0.499755859375f && fabsf(__fsub_rn(q0.y, c.y)) < 0.499755859375f &&
           fabsf(q0.x) <= 512.0f && fabsf(q0.y) <= 512.0f;
    q[i] = __float_as_uint(m.x) - 0x4B400000u;
    q[i + 1] = __float_as_uint(m.y) - 0x4B400000u;
  }
  if (!sure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = (uint32_t)quant_code_fast(x[i], z, s, r, bits, 0);
  }
  if (bits == 8) {
    const uint2 w = make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
    *reinterpret_cast<uint2*>(rec + off + t * D + c0) = w;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= q[2 * j] << (4 * j) | q[2 * j + 1] << (16 + 4 * j);
    *reinterpret_cast<uint32_t*>(rec + off + t * (D / 2) + c0 / 2) = w;
  }
  if ((c0 & ((1 << lg_group) - 1)) == 0) {
    const int g = t * (D >> lg_group) + (c0 >> lg_group);
    store_meta(rec + meta_off, g, 0, 0, z, s);
  }
}

struct AppendRows {
  const void *k, *v;
  long ks, vs;
  int page_bf16, lg_wpt, aligned;
};

template <typename T, int D, bool QUANT>
__global__ void __launch_bounds__(kThreads, QUANT ? 5 : 4) pages_append_kernel(PagesView pv, BatchView bv, RopeView rv, AppendRows a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ Place place[kRowWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nsub = 1 << a.lg_wpt, sub = warp & (nsub - 1), tpb = kRowWarps >> a.lg_wpt;
  const int rg = lane / LPR, c0 = (lane % LPR) * 8, H = pv.heads;
  pdl_wait();
  pdl_trigger();
  for (long t0 = (long)blockIdx.x * tpb; t0 < bv.new_tokens; t0 += (long)gridDim.x * tpb) {
    __syncthreads();
    find_places(pv, bv, &rv, t0, tpb, place);
    const Place p = place[warp >> a.lg_wpt];
    if (p.page < 0) continue;
    const long t = t0 + (warp >> a.lg_wpt);
    const Turn turn = load_turn(rv, p.turn, c0, lane);
    const T* k = static_cast<const T*>(a.k) + t * a.ks;
    const T* v = static_cast<const T*>(a.v) + t * a.vs;
    constexpr int U = QUANT ? 1 : 2;
    for (int h0 = sub * RPW; h0 < H; h0 += nsub * RPW * U) {
      Row8<T> kr[U], vr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = min(h0 + u * nsub * RPW + rg, H - 1);
        kr[u] = load8(k + (long)h * D + c0, a.aligned);
        vr[u] = load8(v + (long)h * D + c0, a.aligned);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hu = h0 + u * nsub * RPW;
        if (hu >= H) break;
        const int h = min(hu + rg, H - 1);
        char* rec = record_of(pv, p.page, h, p.slot);
        float x[8];
        unpack8(kr[u], x);
        turn8(turn, x);
        put8<D, QUANT>(rec, 0, pv.L.km_off, pv.L.k_bits, pv.L.k_lg, p.slot, c0, x, a.page_bf16, hu + rg < H);
        unpack8(vr[u], x);
        put8<D, QUANT>(rec, pv.L.v_off, pv.L.vm_off, pv.L.v_bits, pv.L.v_lg, p.slot, c0, x, a.page_bf16, hu + rg < H);
      }
    }
  }
}

// -------------------------------------------------------------------- read --

// 8 channels of one tensor's row as the page holds them.
template <int BITS>
struct Held8 {
  uint32_t w[BITS / 4];
  uint32_t zs;  // (zero, step) of their group
};

template <int BITS>
__device__ __forceinline__ Held8<BITS> load_held(const char* row, const char* meta) {
  Held8<BITS> x;
  if constexpr (BITS == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(row);
    x.w[0] = w.x, x.w[1] = w.y, x.w[2] = w.z, x.w[3] = w.w;
    x.zs = 0;
  } else {
    if constexpr (BITS == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(row);
      x.w[0] = w.x, x.w[1] = w.y;
    } else {
      x.w[0] = *reinterpret_cast<const uint32_t*>(row);
    }
    x.zs = *reinterpret_cast<const uint32_t*>(meta);
  }
  return x;
}

// zero + code * step, rounded once to fp16
template <int BITS>
__device__ __forceinline__ uint4 held_values(const Held8<BITS>& x) {
  if constexpr (BITS == 16) {
    return make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  } else {
    const __half2 z = __low2half2(as_h2(x.zs)), s = __high2half2(as_h2(x.zs));
    if constexpr (BITS == 8)
      return make_uint4(bytes<0>(x.w[0], s, z), bytes<1>(x.w[0], s, z), bytes<0>(x.w[1], s, z), bytes<1>(x.w[1], s, z));
    else
      return make_uint4(nibbles<0>(x.w[0], s, z), nibbles<1>(x.w[0], s, z), nibbles<2>(x.w[0], s, z), nibbles<3>(x.w[0], s, z));
  }
}

// A warp takes a token's heads, kReadHeads of a lane in flight; what lies in a record does
// not change from head to head, so a head costs four loads, its values and two stores.
// (Offsets worked out head by head took 169 instructions a pass and, in the registers of 8
// CTAs per SM, spills.)  509 pages of 64 tokens, 40 heads of 128, 8- and 4-bit, copied and
// read in four layers, us: that form 1165; now 927 with two heads in flight and 5 CTAs per
// SM, 949 with one and 8, 918 with four and 4, which costs short reads more.
// `turns`: rows that a warp takes one after the other of those whose places are found at
// once.
constexpr int kReadTurns = 8, kReadHeads = 2;

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kThreads, 5) pages_read_kernel(PagesView pv, BatchView bv, char* k_out, char* v_out,
                                                              int lg_wpt, int turns) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kReadHeads;
  __shared__ Place place[kRowWarps * kReadTurns];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nsub = 1 << lg_wpt, sub = warp & (nsub - 1), tpb = kRowWarps >> lg_wpt;
  const int h_first = sub * RPW + lane / LPR, c0 = (lane % LPR) * 8, H = pv.heads, h_step = nsub * RPW;
  const long head_bytes = page_head_bytes(pv), rec_step = h_step * head_bytes;
  pdl_wait();
  pdl_trigger();
  for (long t0 = (long)blockIdx.x * tpb * turns; t0 < bv.new_tokens; t0 += (long)gridDim.x * tpb * turns) {
    __syncthreads();
    find_places(pv, bv, nullptr, t0, tpb * turns, place);
    for (int i = warp >> lg_wpt; i < tpb * turns; i += tpb) {
      const Place p = place[i];
      if (p.page < 0) continue;
      const int t = p.slot & 15;
      const char* rec = record_of(pv, p.page, h_first, p.slot);
      auto row_at = [&](int bits) { return bits == 16 ? (c0 >> 6) * 2048 + t * 128 + ((((c0 >> 3) & 7) ^ (t & 7)) << 4) : t * (D * bits / 8) + c0 * bits / 8; };
      const int k_row = row_at(KB), v_row = pv.L.v_off + row_at(VB);
      const int k_meta = pv.L.km_off + (t * (D >> pv.L.k_lg) + (c0 >> pv.L.k_lg)) * 4;
      const int v_meta = pv.L.vm_off + (t * (D >> pv.L.v_lg) + (c0 >> pv.L.v_lg)) * 4;
      long at = (((t0 + i) * H + h_first) * D + c0) * 2;
      for (int h = h_first; h < H; h += h_step * U) {
        Held8<KB> k[U];
        Held8<VB> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const char* r = rec + u * rec_step;
          if (h + u * h_step < H) {
            if (k_out) k[u] = load_held<KB>(r + k_row, r + k_meta);
            if (v_out) v[u] = load_held<VB>(r + v_row, r + v_meta);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long o = at + (long)u * h_step * (D * 2);
          if (h + u * h_step < H) {
            if (k_out) *reinterpret_cast<uint4*>(k_out + o) = held_values<KB>(k[u]);
            if (v_out) *reinterpret_cast<uint4*>(v_out + o) = held_values<VB>(v[u]);
          }
        }
        rec += U * rec_step;
        at += (long)U * h_step * (D * 2);
      }
    }
  }
}

template <int D>
const void* read_fn(const PagesLayout& L) {
  if (L.k_bits == 16) return (const void*)pages_read_kernel<D, 16, 16>;
  if (L.k_bits == 8) return L.v_bits == 8 ? (const void*)pages_read_kernel<D, 8, 8> : (const void*)pages_read_kernel<D, 8, 4>;
  return L.v_bits == 8 ? (const void*)pages_read_kernel<D, 4, 8> : (const void*)pages_read_kernel<D, 4, 4>;
}

unsigned token_blocks(long tokens, int lg_wpt) {
  const long per = kRowWarps >> lg_wpt;
  return (unsigned)std::min((tokens + per - 1) / per, 152L * 8 * 4);
}

template <typename T, bool QUANT>
const void* append_fn(int D) {
  return D == 64    ? (const void*)pages_append_kernel<T, 64, QUANT>
         : D == 128 ? (const void*)pages_append_kernel<T, 128, QUANT>
                    : (const void*)pages_append_kernel<T, 256, QUANT>;
}
template <typename T>
const void* append_fn(int D, bool quant) {
  return quant ? append_fn<T, true>(D) : append_fn<T, false>(D);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

cudaError_t launch_norm_rope(const kvq_norm_rope_args& x, const RopeView& rv, cudaStream_t st) {
  const int per = x.dtype == KVQ_F32 ? 4 : 8;  // elements of 16 bytes
  NormArgs a = {};
  a.q = x.q, a.k = x.k, a.q_out = x.q_out, a.k_out = x.k_out;
  a.qs = x.q_stride, a.ks = x.k_stride, a.qos = x.q_out_stride, a.kos = x.k_out_stride;
  a.qw = x.q_weight, a.kw = x.k_weight;
  a.tokens = x.tokens, a.q_heads = x.q_heads, a.kv_heads = x.kv_heads, a.norm = x.norm, a.eps = x.eps;
  a.w_f32 = x.weight_dtype == KVQ_F32;
  a.aligned = (!x.q_heads || (aligned16(x.q) && aligned16(x.q_out) && x.q_stride % per == 0 && x.q_out_stride % per == 0)) &&
              (!x.kv_heads || (aligned16(x.k) && aligned16(x.k_out) && x.k_stride % per == 0 && x.k_out_stride % per == 0));
  a.w_aligned = aligned16(x.q_weight) && aligned16(x.k_weight);
  if (x.dtype == KVQ_F32) return launch_norm_t<float>(x, rv, a, st);
  if (x.dtype == KVQ_BF16) return launch_norm_t<__nv_bfloat16>(x, rv, a, st);
  return launch_norm_t<__half>(x, rv, a, st);
}

cudaError_t launch_pages_append(const PagesView& pv, const BatchView& bv, const RopeView& rv, const void* k,
                                const void* v, int in_dtype, int page_bf16, long k_stride, long v_stride,
                                cudaStream_t st) {
  const int per = in_dtype == KVQ_F32 ? 4 : 8;
  const int rpw = 32 / (pv.head_dim / 8);
  AppendRows a = {k, v, k_stride, v_stride, page_bf16, 0, 0};
  a.aligned = aligned16(k) && aligned16(v) && k_stride % per == 0 && v_stride % per == 0;
  a.lg_wpt = lg_warps_per_token(bv.new_tokens, (pv.heads + rpw - 1) / rpw);
  PagesView p = pv;
  BatchView b = bv;
  RopeView r = rv;
  void* args[] = {&p, &b, &r, &a};
  const bool quant = pv.L.k_bits != 16;
  const void* fn = in_dtype == KVQ_F32    ? append_fn<float>(pv.head_dim, quant)
                   : in_dtype == KVQ_BF16 ? append_fn<__nv_bfloat16>(pv.head_dim, quant)
                                          : append_fn<__half>(pv.head_dim, quant);
  return launch_pdl(fn, dim3(token_blocks(bv.new_tokens, a.lg_wpt)), dim3(kThreads), 0, st, args);
}

cudaError_t launch_pages_read(const PagesView& pv, const BatchView& bv, void* k_out, void* v_out, cudaStream_t st) {
  const int rpw = 32 / (pv.head_dim / 8);
  int lg = lg_warps_per_token(bv.new_tokens, (pv.heads + rpw - 1) / rpw);
  PagesView p = pv;
  BatchView b = bv;
  char *ko = static_cast<char*>(k_out), *vo = static_cast<char*>(v_out);
  const long per = kRowWarps >> lg;
  int turns = 1;  // (doubled while the blocks fill the card twice)
  while (turns < kReadTurns && bv.new_tokens >= per * turns * 2 * 152 * 8 * 2) turns *= 2;
  void* args[] = {&p, &b, &ko, &vo, &lg, &turns};
  const void* fn = pv.head_dim == 64 ? read_fn<64>(pv.L) : pv.head_dim == 128 ? read_fn<128>(pv.L) : read_fn<256>(pv.L);
  return launch_pdl(fn, dim3(token_blocks((bv.new_tokens + turns - 1) / turns, lg)), dim3(kThreads), 0, st, args);
}

}  // namespace kvq
