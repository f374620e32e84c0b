// kvq_pages_rows.cuh — paged attention for few query rows per kv head (single
// tokens, drafted tokens, short chunks): bound by reading the cache once.
//
// A CTA of four warps walks its units of 64 or 128 tokens; each warp takes a
// quarter, one or two records, brought by bulk copies into the warp's own ring
// of stages, and runs an independent softmax over its tokens, so nothing but the
// end of an item synchronises the warps.  Query rows are the 8 columns of
// m16n8k16 (NM tiles of them), so all query heads of a kv head and several new
// tokens share one read of the cache; keys and values are its left operand, the
// weights are turned by an 8x8 transpose for the second product, and a row's
// maximum, whose tokens lie in eight lanes, is exchanged only where it grows.
//  - 16-bit pages: ldmatrix reads keys and (transposed) values straight from
//    the swizzled rows.
//  - codes: the contraction does not care about the order of channels, tokens
//    or output channels, so each lane is given runs that are contiguous in
//    memory: keys, channels t*D/4 .. of token (g>>1) + 4*(g&1) (g = lane / 4, t =
//    lane % 4); values, channels g*D/8 .. of tokens
//    t, t+4, t+8, t+12.  Each run lies in one group (or two), so a lane needs
//    one (zero, step) per token.  Codes become fp16 by an or with 1024's bits
//    and one exact subtraction; zero + code * step is one fp16 fma, the value
//    that the page stands for.
// Scores, maxima, sums and outputs are fp32.  Weights enter the value product
// as p * 2^7 with a maximum that lags by up to 2^8, so that fp16 weights stay
// normal down to 2^-21 of the largest.  Over 16-bit pages the weights of a sequence
// of up to 16 rows (of any at head_dim 256) are split into the operand type and its
// remainder (a second product, hidden behind the reads); elsewhere they are rounded
// to the operand type (fp16, or bf16 for bf16 pages), which adds about as much to
// the error as the output's own rounding does.  The sequence's own rows decide, not
// the kernel's: its error does not depend on its neighbours in the batch.
//
// Measured: 16 sequences of 4113 bf16 tokens, 40 heads of 128: 207 us, 96 % of a
// copy's bandwidth.  64 sequences of 1k to 32k 4-bit tokens, 32 query heads over 8
// of 128: 310 us, 60 % (375 with 16 rows and three CTAs per SM in place of 8 and
// four; 330 with 8 rows and five CTAs): a record of codes costs about as many
// instructions whatever the rows are, and fixed-latency waits take the slots that
// are left.  5 drafted tokens, 20 rows, over 8-bit pages: 59 us (floor 29), two
// CTAs per SM; 66 as two 16-row operands.  (That form, the rows as the left
// operand, was 90 us against 99 for a full 32 rows of 32 sequences of 4096 4-bit
// tokens, heads of 128, but 88 against 71 for 16 and 86 against 56 for 8.)
// 8 sequences of 2048 fp16 tokens, 12 heads of 64: 15 us in a graph, of which 9 are
// launch, plan and join.
#pragma once

#include <cfloat>

#include "kvq_pages_attn.cuh"

namespace kvq {

constexpr int kRowsWarps = 4;
constexpr int kSplitRows = 16;  // most rows of a sequence whose weights the 24- and 32-row kernels split

template <int FMT>
struct Fmt {
  static constexpr int KB = FMT <= kFmtBf16 ? 16 : (FMT == kFmt88 || FMT == kFmt84 ? 8 : 4);
  static constexpr int VB = FMT <= kFmtBf16 ? 16 : (FMT == kFmt88 || FMT == kFmt48 ? 8 : 4);
  static constexpr bool kBf16 = FMT == kFmtBf16;
  static constexpr bool kQuant = KB < 16;
};

template <int D, int FMT, int NM>
struct RowsCfg {
  using F = Fmt<FMT>;
  static constexpr int ROWS = 8 * NM;
  // a record with the most metadata (groups of 32)
  static constexpr int REC = 2 * D * (F::KB + F::VB) + (F::kQuant ? 2 * 16 * (D / 32) * 4 : 0);
  // CTAs per SM that registers and shared memory are cut for (a few bytes a sequence
  // come on top: 1024 sequences can cost one of them)
  static constexpr int CTAS = D == 64    ? (NM <= 2 ? 4 : 3)
                              : D == 128 ? (F::kQuant && NM <= 2 ? 5 - NM : 2)
                                         : (!F::kQuant ? 1 : (NM == 1 && F::KB + F::VB < 16 ? 3 : 2));
  static constexpr int BUDGET = CTAS == 4 ? 12544 : (CTAS == 3 ? 16384 : 24576);  // bytes of a warp's ring
  // records of a warp's step and stage: two where two such stages fit, so that
  // the softmax's exchanges and the loop cost half as much per token
  static constexpr int RECS = 4 * REC > BUDGET ? 1 : 2;
  static constexpr int STEP = 16 * RECS, BK = STEP * kRowsWarps;  // tokens of a step and of a unit
  static constexpr int STAGE = RECS * REC;
  static constexpr int NS = BUDGET / STAGE < 2 ? 2 : (BUDGET / STAGE > 4 ? 4 : BUDGET / STAGE);
  // Weights as operand + remainder: always, or for sequences of up to kSplitRows rows
  static constexpr bool kSplit = !F::kQuant, kSplitSome = kSplit && ROWS > kSplitRows;
  static constexpr int RING = kRowsWarps * NS * STAGE;
  static constexpr int MERGE = kRowsWarps * ROWS * (D + 2) * 4;
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE);
  // (the queries and little else are static; 1 KB of a CTA is the system's)
  static_assert(CTAS * (SMEM + NM * (D / 16) * 256 + 2048) <= 228 * 1024, "CTAs of an SM fit its shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(x) : "r"(a) : "memory");
  return x;
}
// N 32-bit words from shared memory, in the widest loads
template <int N>
__device__ __forceinline__ void ldsv(uint32_t a, uint32_t* x) {
  if (N == 1) {
    x[0] = lds32(a);
  } else if (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(x[0]), "=r"(x[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                   : "=r"(x[4 * i]), "=r"(x[4 * i + 1]), "=r"(x[4 * i + 2]), "=r"(x[4 * i + 3])
                   : "r"(a + 16 * i)
                   : "memory");
  }
}
// Two codes -> zero + code * step: the codes' bits or-ed into the mantissas of a
// power of two give power + code exactly, the power is taken off exactly, and
// one fma rounds.
__device__ __forceinline__ uint32_t dequant2(uint32_t biased, uint32_t power, __half2 s, __half2 z) {
  return as_u32(__hfma2(__hsub2(as_h2(biased), as_h2(power)), s, z));
}
// nibble J of both halves: bits 0..3 under 1024 (0x6400), bits 4..7 under 64 (0x5400)
template <int J>
__device__ __forceinline__ uint32_t nibbles(uint32_t x, __half2 s, __half2 z) {
  const uint32_t y = J >= 2 ? x >> 8 : x;
  return (J & 1) ? dequant2(lop3_and_or(y, 0x00f000f0u, 0x54005400u), 0x54005400u, s, z)
                 : dequant2(lop3_and_or(y, 0x000f000fu, 0x64006400u), 0x64006400u, s, z);
}
// the low / high two of four 8-bit codes
template <int HIGH>
__device__ __forceinline__ uint32_t bytes(uint32_t x, __half2 s, __half2 z) {
  return dequant2(__byte_perm(x, 0x64646464u, HIGH ? 0x4342 : 0x4140), 0x64006400u, s, z);
}

// Byte offsets inside a record that a lane reads from, fixed for the launch.
template <int D, int FMT>
struct LaneOffsets {
  uint32_t k, v;    // key / value rows of its first token
  uint32_t km, vm;  // their metadata
  uint32_t km8, vm4;  // metadata of 8 / 4 tokens
  __device__ __forceinline__ LaneOffsets(const PagesLayout& L, int lane) {
    using F = Fmt<FMT>;
    const int g = lane >> 2, t = lane & 3;
    if constexpr (!F::kQuant) {
      k = ((lane & 7) + ((lane >> 4) << 3)) * 128;
      v = L.v_off + ((lane & 7) + (((lane >> 3) & 1) << 3)) * 128;
      km = vm = km8 = vm4 = 0;
    } else {
      const int tok = (g >> 1) + 4 * (g & 1);
      k = tok * (D * F::KB / 8) + t * (D / 4 * F::KB / 8);
      v = L.v_off + t * (D * F::VB / 8) + g * (D / 8 * F::VB / 8);
      km = L.km_off + (tok * (D >> L.k_lg) + ((t * (D / 4)) >> L.k_lg)) * 4;
      vm = L.vm_off + (t * (D >> L.v_lg) + ((g * (D / 8)) >> L.v_lg)) * 4;
      km8 = 8 * (D >> L.k_lg) * 4;
      vm4 = 4 * (D >> L.v_lg) * 4;
    }
  }
};

// One 16-token record's scores: acc[m] += K Q_m^T.  sq: the query operands in
// shared memory, [m][mma step][lane] of two words.
template <int D, int FMT, int NM>
__device__ __forceinline__ void rows_scores(uint32_t st, const PagesLayout& L, const LaneOffsets<D, FMT>& lo,
                                            uint32_t sq, int lane, float (*acc)[4]) {
  using F = Fmt<FMT>;
  const uint32_t qa = sq + lane * 8;
  // keys of tokens 0..7 and 8..15 (two words each) of a step
  auto step = [&](int ks, const uint32_t* b0, const uint32_t* b1) {
    const uint32_t k[4] = {b0[0], b1[0], b0[1], b1[1]};
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      uint32_t q[2];
      ldsv<2>(qa + (m * (D / 16) + ks) * 256, q);
      mma16<F::kBf16>(acc[m], k, q[0], q[1]);
    }
  };
  if constexpr (!F::kQuant) {
    const uint32_t base = st + lo.k, turn = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b[4];
      ldsm4(base + (ks >> 2) * 2048 + (turn ^ ((2 * ks & 7) << 4)), b);
      step(ks, b, b + 2);
    }
  } else {
    constexpr int SPAN = D / 4;               // channels a lane reads of a token
    constexpr int RUN = SPAN < 32 ? SPAN : 32;  // channels in one group at least
    constexpr int W = RUN * F::KB / 32;       // words of a run
    const uint32_t row = st + lo.k, meta = st + lo.km;
#pragma unroll
    for (int r = 0; r < SPAN / RUN; ++r) {
      uint32_t w[2][W];
      __half2 z[2], s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a lane's run r starts at its span's start: the span is a whole number of groups, or inside one)
        const __half2 zs = as_h2(lds32(meta + h * lo.km8 + (r ? ((r * RUN) >> L.k_lg) * 4 : 0)));
        z[h] = __low2half2(zs), s[h] = __high2half2(zs);
        ldsv<W>(row + h * (D * F::KB) + r * (RUN * F::KB / 8), w[h]);
      }
#pragma unroll
      for (int i = 0; i < RUN / 4; ++i) {  // one mma step: 4 channels
        uint32_t b[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (F::KB == 8) {
            b[h][0] = bytes<0>(w[h][i], s[h], z[h]);
            b[h][1] = bytes<1>(w[h][i], s[h], z[h]);
          } else if (i & 1) {
            b[h][0] = nibbles<2>(w[h][i / 2], s[h], z[h]);
            b[h][1] = nibbles<3>(w[h][i / 2], s[h], z[h]);
          } else {
            b[h][0] = nibbles<0>(w[h][i / 2], s[h], z[h]);
            b[h][1] = nibbles<1>(w[h][i / 2], s[h], z[h]);
          }
        }
        step(r * (RUN / 4) + i, b[0], b[1]);
      }
    }
  }
}

// o[m][16 channels] += V^T P_m^T of one record, m < NM; p: the weights as operands,
// rest: their remainders (SPLIT).
template <int D, int FMT, int NM, bool SPLIT>
__device__ __forceinline__ void rows_values(uint32_t st, const LaneOffsets<D, FMT>& lo, const uint32_t (*p)[2],
                                            const uint32_t (*rest)[2], int lane, float (*o)[D / 16][4]) {
  using F = Fmt<FMT>;
  // channels 0..7 and 8..15 of step j: values of tokens 0..7 and 8..15 (a word each)
  auto step = [&](int j, const uint32_t* b0, const uint32_t* b1) {
    const uint32_t v[4] = {b0[0], b1[0], b0[1], b1[1]};
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      mma16<F::kBf16>(o[m][j], v, p[m][0], p[m][1]);
      if constexpr (SPLIT) mma16<F::kBf16>(o[m][j], v, rest[m][0], rest[m][1]);
    }
  };
  if constexpr (!F::kQuant) {
    const uint32_t base = st + lo.v, turn = ((lane >> 4) ^ (lane & 7)) << 4;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t b[4];
      ldsm4t(base + (j >> 2) * 2048 + (turn ^ ((2 * j & 7) << 4)), b);
      step(j, b, b + 2);
    }
  } else {
    constexpr int RUN = D / 8;           // channels a lane reads of a token
    constexpr int W = RUN * F::VB / 32;  // words of them
    uint32_t w[4][W];
    __half2 zs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      zs[j] = as_h2(lds32(st + lo.vm + j * lo.vm4));
      ldsv<W>(st + lo.v + j * (4 * D * F::VB / 8), w[j]);
    }
    __half2 z[2], s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      z[h] = __lows2half2(zs[2 * h], zs[2 * h + 1]);
      s[h] = __highs2half2(zs[2 * h], zs[2 * h + 1]);
    }
    if (F::VB == 8) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        uint32_t x[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h][0] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x5140);
          x[h][1] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x7362);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t b0[2] = {bytes<0>(x[0][c], s[0], z[0]), bytes<0>(x[1][c], s[1], z[1])};
          const uint32_t b1[2] = {bytes<1>(x[0][c], s[0], z[0]), bytes<1>(x[1][c], s[1], z[1])};
          step(2 * i + c, b0, b1);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        uint32_t x[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h][0] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x5410);
          x[h][1] = __byte_perm(w[2 * h][i], w[2 * h + 1][i], 0x7632);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t b[2][2];
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              b[y][h] = c == 0   ? nibbles<0>(x[h][y], s[h], z[h])
                        : c == 1 ? nibbles<1>(x[h][y], s[h], z[h])
                        : c == 2 ? nibbles<2>(x[h][y], s[h], z[h])
                                 : nibbles<3>(x[h][y], s[h], z[h]);
          step(4 * i + c, b[0], b[1]);
        }
      }
    }
  }
}

// E so that m * 2^E lies in [2^14, 2^15), for every float; 0 for m = 0.
__device__ __forceinline__ int query_exp(float m) {
  if (!(m > 0.0f)) return 0;
  const bool tiny = m < FLT_MIN;  // (below the normal range the exponent's bits are zero)
  return 14 + 127 - ((__float_as_int(tiny ? m * 0x1p64f : m) >> 23) & 0xff) + (tiny ? 64 : 0);
}

// What the scores of a row scaled by 2^E are to be multiplied by; never zero, which
// would turn a hidden score's -inf into NaN.
__device__ __forceinline__ float row_factor(const AttnArgs& a, int E) {
  return fmaxf(a.scale_log2 * exp2i(-(E / 2)) * exp2i(-(E - E / 2)), FLT_MIN);
}

// Row tile m of a piece's queries as A operands in shared memory (one warp), and
// what its rows' scores are to be multiplied by.  Over codes q becomes fp16: a
// bf16 row is scaled by the power of two that puts its largest magnitude in
// [2^14, 2^15), so that nothing overflows and its 8 significant bits survive
// down to 2^-28 of the largest, wherever in bf16's range that lies (E is 147 for its
// smallest number).
template <int D, int FMT>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Piece& p, int m, int lane, uint32_t sq, float* sc) {
  using F = Fmt<FMT>;
  const int g = lane >> 2, t = lane & 3;
  uint32_t q[D / 16][2];
  const int r = p.r0 + min(m * 8 + g, p.rows - 1);
  const uint16_t* row = static_cast<const uint16_t*>(a.q) + (long)(p.s.s0 + r / a.rep) * a.q_stride +
                        (long)(p.head * a.rep + r % a.rep) * D;
  auto pair = [&](int c) -> uint32_t {
    if (a.q_aligned) return *reinterpret_cast<const uint32_t*>(row + c);
    return (uint32_t)row[c] | (uint32_t)row[c + 1] << 16;
  };
  float f = a.scale_log2;
  if constexpr (!F::kQuant) {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      q[ks][0] = pair(ks * 16 + 2 * t);
      q[ks][1] = pair(ks * 16 + 8 + 2 * t);
    }
  } else {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      q[ks][0] = pair(t * (D / 4) + 4 * ks);
      q[ks][1] = pair(t * (D / 4) + 4 * ks + 2);
    }
    if (a.q_bf16) {
      float mx = 0.0f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = q[ks][i];
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int E = query_exp(mx);
      // 2^E in two factors: E may pass the range of one float
      const float f0 = exp2i(E / 2), f1 = exp2i(E - E / 2);
      f = row_factor(a, E);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = q[ks][i];
          q[ks][i] = pack2<false>(__uint_as_float(w << 16) * f0 * f1, __uint_as_float(w & 0xffff0000u) * f0 * f1);
        }
    }
  }
  if (t == 0) sc[m * 8 + g] = f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};\n" ::"r"(sq + (m * (D / 16) + ks) * 256 + lane * 8), "r"(q[ks][0]), "r"(q[ks][1])
                 : "memory");
}

// (out of line: it is rarely taken, and its registers are not the loop's)
static __device__ __noinline__ bool rows_wait_slow(uint32_t bar, int phase, int* dead, int* err) {
  return cta_wait(bar, phase, dead, err);
}

// MASK: rows see what a.seen says (trees of drafted tokens) or everything (cross
// attention) in place of what lies before them.
template <int D, int FMT, int NM, bool MASK>
__global__ void __launch_bounds__(kRowsWarps * 32, RowsCfg<D, FMT, NM>::CTAS) pages_rows_kernel(const __grid_constant__ AttnArgs a) {
  using C = RowsCfg<D, FMT, NM>;
  using F = Fmt<FMT>;
  constexpr int ROWS = C::ROWS, NS = C::NS, BK = C::BK, RECS = C::RECS, STEP = C::STEP;
  extern __shared__ __align__(1024) char smem[];
  __shared__ Work<BK, ROWS> work;
  __shared__ Piece piece;
  __shared__ float row_scale[ROWS];
  __shared__ __align__(16) uint32_t queries[NM * (D / 16) * 64];
  __shared__ __align__(8) uint64_t bars[kRowsWarps * NS];
  __shared__ int dead;  // a wait gave up: the CTA leaves
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const int g = lane >> 2, t = lane & 3;
  const LaneOffsets<D, FMT> offs(a.pv.L, lane);
  const uint32_t sq = smem_u32(queries);
  const uint32_t ring = smem_u32(smem) + warp * NS * C::STAGE;
  const uint32_t bar = smem_u32(bars) + warp * NS * 8;
  if (lane < NS) mbar_init(bar + lane * 8, 1);
  if (threadIdx.x == 0) dead = 0;
  fence_mbar_init();
  pdl_wait();
  plan_work<BK, ROWS, true, MASK>(a, &work, reinterpret_cast<long*>(smem + C::SMEM));
  pdl_trigger();
  if (cta >= work.ctas) {
    if (threadIdx.x == 0) a.split[cta].parts = 0;
    return;
  }
  long u = work.own ? 0 : cta_begin(&work, cta);
  const long end = work.own ? 1 : cta_begin(&work, cta + 1);
  int stage = 0, phase = 0;  // of the next tile to be read; the ring is empty between pieces
  bool joined = false;
  while (u < end) {
    if (warp == 0) {
      const Piece x = work.own ? own_piece<MASK>(a, &work, cta) : find_piece<MASK>(a, &work, u, end);
      if (lane == 0) piece = x;
    }
    __syncthreads();
    const Piece p = piece;
    u += work.own ? 1 : p.nblk;
    // this warp's steps: STEP tokens at 4 * block + warp, while they hold a visible one
    const int see1 = MASK ? p.s.len : max(p.s.p0 + (p.r0 + p.rows - 1) / a.rep + 1, 0);
    const int see0 = a.window > 0 ? max(p.s.p0 + (MASK ? 0 : p.r0 / a.rep) - a.window + 1, 0) : 0;
    const int tok0 = (p.blk * kRowsWarps + warp) * STEP;  // of step j: tok0 + BK * j
    int j = 0;
    const int nt = max(min((see1 - tok0 + BK - 1) / BK, p.nblk), 0);
    if (j < nt && tok0 + STEP <= see0) ++j;

    // Copies of a step into stage s: lane r % RECS brings record r % RECS, if it
    // holds a token of the sequence.  The first NS steps at once, RECS lanes each.
    const PageRun run(a.pv, p.head);
    auto bring = [&](int tok, int page, int s) {
      const int rec = lane % RECS;
      const bool second = RECS == 2 && tok - rec * 16 + 16 < p.s.len;
      if (rec == 0) mbar_expect(bar + s * 8, second ? 2 * a.pv.L.tile_bytes : a.pv.L.tile_bytes);
      if (rec == 0 || second)
        bulk_load(ring + s * C::STAGE + rec * C::REC, run.at(a, page, tok), a.pv.L.tile_bytes, bar + s * 8);
    };
    auto page_of = [&](int tok) { return tok < p.s.len ? page_index(a, p.b, tok) : 0; };
    if (lane < RECS * min(NS, nt - j)) {
      const int tok = tok0 + BK * (j + lane / RECS) + (lane % RECS) * 16;
      int s = stage + lane / RECS;
      s = s >= NS ? s - NS : s;
      bring(tok, page_of(tok), s);
    }
    __syncwarp();
    int next = lane < RECS && j + NS < nt ? page_of(tok0 + BK * (j + NS) + lane * 16) : 0;

    if (warp < NM) load_queries<D, FMT>(a, p, warp, lane, sq, row_scale);
    __syncthreads();
    auto row_at = [&](int m, int e) { return m * 8 + 2 * t + e; };  // a lane's two rows of a tile
    float sc[NM][2];
    float o[NM][D / 16][4], mx[NM][2], sum[NM][2];
    int pos[NM][2];  // the rows' positions; MASK: their tokens among the call's
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][i][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[m][e] = -INFINITY;
        sum[m][e] = 0.0f;
        sc[m][e] = row_scale[row_at(m, e)];
        pos[m][e] = (MASK ? p.s.s0 : p.s.p0) + (p.r0 + min(row_at(m, e), p.rows - 1)) / a.rep;
      }
    }
    // the rows' first and last position: steps between need no mask
    const int pos_lo = MASK ? p.s.p0 - 1 : p.s.p0 + p.r0 / a.rep;
    const int pos_hi = MASK ? p.s.len - 1 : p.s.p0 + (p.r0 + p.rows - 1) / a.rep;
    constexpr int SPLIT_NM = NM < kSplitRows / 8 ? NM : kSplitRows / 8;  // row tiles that are split
    const bool split = C::kSplit && (!C::kSplitSome || p.s.n * a.rep <= kSplitRows);

    for (; j < nt; ++j) {
      const bool here = mbar_try(bar + stage * 8, phase) || rows_wait_slow(bar + stage * 8, phase, &dead, a.pv.err);
      if (!__all_sync(0xffffffffu, here)) {  // (each lane has its own clock; the warp decides together)
        ring_drain<NS>(bar, stage, phase, min(NS, nt - j));
        break;
      }
      const uint32_t st = ring + stage * C::STAGE;
      const int tok = tok0 + BK * j;
      if (tok + STEP > p.s.len) {  // the sequence ends inside this step: what lies behind has no effect
        const int n = p.s.len - tok;
        if (!F::kQuant) {
          for (int i = lane; i < (STEP - n) * (D / 8); i += 32) {
            const int r = n + i / (D / 8), c = i % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(st + (r >> 4) * C::REC + a.pv.L.v_off + (c >> 3) * 2048 + (r & 15) * 128 + ((c & 7) << 4)),
                         "r"(0)
                         : "memory");
          }
        } else {
          const int per = D >> a.pv.L.v_lg;
          for (int i = lane; i < (STEP - n) * per; i += 32) {
            const int r = n + i / per, c = i % per;
            asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(st + (r >> 4) * C::REC + a.pv.L.vm_off + ((r & 15) * per + c) * 4), "r"(0)
                         : "memory");
          }
        }
        fence_async();
        __syncwarp();
      }
      float acc[RECS][NM][4];  // [2 h + e]: the lane's token h, its row e
#pragma unroll
      for (int x = 0; x < RECS; ++x) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[x][m][e] = 0.0f;
        rows_scores<D, FMT, NM>(st + x * C::REC, a.pv.L, offs, sq, lane, acc[x]);
      }
      const bool edge = tok + STEP - 1 > pos_lo || (a.window > 0 && tok <= pos_hi - a.window);
      bool grow = false;
      float top[NM][2];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        if (edge) {
          uint32_t vis[2] = {};
          if constexpr (MASK) {
#pragma unroll
            for (int e = 0; e < 2; ++e) vis[e] = seen_bits(a, p.s, pos[m][e], tok);
          }
#pragma unroll
          for (int x = 0; x < RECS; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int in = 16 * x + 8 * (e >> 1) + (F::kQuant ? (g >> 1) + 4 * (g & 1) : g);  // token of the step
              const int c = tok + in, at = pos[m][e & 1];
              const bool hidden = MASK ? !(vis[e & 1] >> in & 1) : c > at || (a.window > 0 && c <= at - a.window);
              if (hidden) acc[x][m][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int y = 0; y < RECS; ++y) x = fmaxf(fmaxf(x, acc[y][m][e]), acc[y][m][2 + e]);
          top[m][e] = x * sc[m][e];
          grow = grow || top[m][e] > mx[m][e] + 8.0f;
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (a row's tokens lie in eight lanes; only now do they have to agree)
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top[m][e] = fmaxf(top[m][e], __shfl_xor_sync(0xffffffffu, top[m][e], w));
            const float to = fmaxf(mx[m][e], top[m][e]);
            const float f = to == -INFINITY ? 1.0f : fast_exp2(mx[m][e] - to);
            mx[m][e] = to;
            sum[m][e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[m][i][e] *= f;
              o[m][i][2 + e] *= f;
            }
          }
      }
#pragma unroll
      for (int x = 0; x < RECS; ++x) {
        uint32_t pa[NM][2], pr[SPLIT_NM][2];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          const float b0 = mx[m][0] == -INFINITY ? 0.0f : mx[m][0] - 7.0f;
          const float b1 = mx[m][1] == -INFINITY ? 0.0f : mx[m][1] - 7.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float u = fast_exp2(fmaf(acc[x][m][2 * h], sc[m][0], -b0));
            const float v = fast_exp2(fmaf(acc[x][m][2 * h + 1], sc[m][1], -b1));
            sum[m][0] += u;
            sum[m][1] += v;
            const uint32_t w = pack2<F::kBf16>(u, v);
            pa[m][h] = transpose8x8(w);
            if (split && m < SPLIT_NM) {
              float2 back;
              if (F::kBf16) back = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
              else back = __half22float2(as_h2(w));
              pr[m][h] = transpose8x8(pack2<F::kBf16>(u - back.x, v - back.y));
            }
          }
        }
        if (split) rows_values<D, FMT, SPLIT_NM, true>(st + x * C::REC, offs, pa, pr, lane, o);
        else rows_values<D, FMT, NM, false>(st + x * C::REC, offs, pa, pr, lane, o);
      }
      fence_async();  // the step's reads (and cleared rows) before the copy into the same bytes
      __syncwarp();
      if (lane < RECS && j + NS < nt) {
        const int tn = tok + BK * NS + lane * 16;
        bring(tn, next, stage);
        if (j + NS + 1 < nt) next = page_of(tn + BK);
      }
      __syncwarp();
      if (++stage == NS) stage = 0, phase ^= 1;
    }

    // ---- merge the four warps
    __syncthreads();
    if (*(volatile int*)&dead) break;
    float* mo = reinterpret_cast<float*>(smem);                 // [warp][ROWS][D]
    float* ml = mo + kRowsWarps * ROWS * D;                     // [warp][ROWS][2]
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = sum[m][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const int r = warp * ROWS + row_at(m, e);
        if (g == 0) ml[2 * r] = mx[m][e], ml[2 * r + 1] = s;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = F::kQuant ? g * (D / 8) + 2 * i : 16 * i + g;
          mo[r * D + c] = o[m][i][e];
          mo[r * D + c + (F::kQuant ? 1 : 8)] = o[m][i][2 + e];
        }
      }
    __syncthreads();
    const bool whole = p.has_first && p.has_last;
    const long slot = (long)cta * 2 + (p.has_first ? 1 : 0);
    for (int i = threadIdx.x; i < p.rows * (D / 4); i += kRowsWarps * 32) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float M = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, ml[2 * (w * ROWS + r)]);
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float m = ml[2 * (w * ROWS + r)];
        const float f = m == -INFINITY ? 0.0f : fast_exp2(m - M);
        const float4 x = *reinterpret_cast<const float4*>(mo + (w * ROWS + r) * D + c);
        l += f * ml[2 * (w * ROWS + r) + 1];
        y.x += f * x.x, y.y += f * x.y, y.z += f * x.z, y.w += f * x.w;
      }
      if (whole) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const int R = p.r0 + r;
        const long at = ((long)(p.s.s0 + R / a.rep) * a.q_heads + p.head * a.rep + R % a.rep) * D + c;
        store_out2(a, at, y.x * inv, y.y * inv);
        store_out2(a, at + 2, y.z * inv, y.w * inv);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * ROWS + r) * D + c) = y;
        if (c == 0) *reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + r) * 2) = make_float2(M, l);
      }
    }
    if (threadIdx.x == 0 && p.has_first && !p.has_last) {
      SplitHead h = {};
      h.parts = p.parts ? p.parts : cta_of(&work, p.item1 - 1) - cta + 1;
      h.rows = p.rows, h.row0 = p.r0, h.q_row = p.s.s0, h.head = p.head;
      a.split[cta] = h;
      joined = true;
    }
    fence_async();  // the merge's plain accesses before the next piece's copies
    __syncthreads();
  }
  if (threadIdx.x == 0 && !joined) a.split[cta].parts = 0;
}

template <int D, int FMT, bool MASK>
AttnKernel rows_kernel_fmt(int nm) {
#define KVQ_ROWS(n) \
  if (nm == n) return {(const void*)pages_rows_kernel<D, FMT, n, MASK>, (size_t)RowsCfg<D, FMT, n>::SMEM, kRowsWarps * 32, 0, 0, 0};
  if constexpr (D <= 128) {
    KVQ_ROWS(4)
    KVQ_ROWS(3)
  }
  KVQ_ROWS(2)
  KVQ_ROWS(1)
#undef KVQ_ROWS
  return {};
}
template <int D, bool MASK>
AttnKernel rows_kernel_dim(int fmt, int nm) {
  switch (fmt) {
    case kFmtF16: return rows_kernel_fmt<D, kFmtF16, MASK>(nm);
    case kFmtBf16: return rows_kernel_fmt<D, kFmtBf16, MASK>(nm);
    case kFmt88: return rows_kernel_fmt<D, kFmt88, MASK>(nm);
    case kFmt44: return rows_kernel_fmt<D, kFmt44, MASK>(nm);
    case kFmt84: return rows_kernel_fmt<D, kFmt84, MASK>(nm);
    default: return rows_kernel_fmt<D, kFmt48, MASK>(nm);
  }
}

}  // namespace kvq
