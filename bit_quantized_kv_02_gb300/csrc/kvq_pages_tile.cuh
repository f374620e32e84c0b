// kvq_pages_tile.cuh — paged attention for many query rows per kv head (chunks
// and prompts): bound by the tensor cores.
//
// One persistent CTA per SM takes its share of the units (blocks of 128
// tokens).  Query rows are (token, head of the group) pairs, so one read of a
// block serves every query head of the kv head; a CTA holds NT tiles of 128
// rows (two, or one at head_dim 256, where the accumulator alone takes half of
// the tensor memory).  Roles of the warps:
//  - loader (16-bit pages): bulk copies of the records' halves into K and V
//    stages; pages are stored in the operand layout, so no tensor map and no
//    shuffling is needed;
//  - raw loaders and dequantizers (codes): one warp per tensor copies records
//    into a ring, two warps per tensor (four with one row tile) turn their codes
//    into fp16 operand tiles (the value the page stands for, one rounding);
//  - one warp issues the matrix instructions: S = Q K^T (both from shared
//    memory), O += P V (P from tensor memory, over the scores it came from);
//  - softmax: a warpgroup per tile, a thread per row, so maxima and sums need
//    no exchange; scores are read from tensor memory once, weights are written
//    back as the operand type.  The running maximum is only raised when a score
//    passes it by 2^8 (then O is rescaled in tensor memory): most blocks leave
//    it alone.  With two tiles the tensor cores work on one while the other's
//    softmax runs; with one, the scores are double-buffered instead;
//  - a scheduler finds the pieces of items ahead of the others.
// Scores, maxima, sums and O are fp32; weights are rounded once to the operand
// type (p * 2^7, as in the few-rows kernel).
//
// Measured: 2048 new tokens at 30720, 32 query heads over 8 of 128, bf16 pages:
// 818 to 833 us on different cards, 1.3 PFLOP/s (66 % of a large library product).
// A CTA takes 418 blocks of two tiles, so a block takes 1.97 us, of which its
// products would take 1.30 at the library product's rate: a tile's chain of scores,
// softmax, value product and the signals between them is what is left (tensor pipe
// active 54 % on a chunk half as long).  509 tokens at 130563, 16 query heads over 2
// of 256, 4-bit keys and 8-bit values: 1444 us, 0.75 PFLOP/s (tensor pipe 29 % at
// 16000), bound by the dequantizers (each CTA turns every code for 128 rows).  Prompts
// of up to 2048 tokens, 40 heads of 128, window 1024: 367 us, tensor pipe 25 %.  A CTA
// has 68 blocks there, in 10.5 pieces, which would take 134 us at the chunk's pace;
// the rest (queries and outputs that no other piece covers, blocks with a mask, a
// second read of the scores in each piece's first block) was not measured apart.
#pragma once

#include "kvq_pages_attn.cuh"
#include "kvq_pages_rows.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

template <int D, int FMT>
struct TileCfg {
  using F = Fmt<FMT>;
  static constexpr int NT = D == 256 ? 1 : 2;      // row tiles of 128
  static constexpr int ROWS = 128 * NT;
  static constexpr int BK = 128;                   // tokens of a block
  static constexpr int NS = D == 256 ? 1 : (D == 128 ? 2 : 3);  // K stages, V stages
  static constexpr int TILE = 128 * D * 2;         // bytes of a Q, K or V tile
  static constexpr int Q_OFF = 0, K_OFF = NT * TILE, V_OFF = K_OFF + NS * TILE;
  // over codes, rings of raw records come behind the tiles, as deep as the 227 KB
  // of a CTA allow (a.ring records per tensor)
  static constexpr int RAW_OFF = V_OFF + NS * TILE;
  static constexpr int SMEM = RAW_OFF + 1024;  // + alignment of the tiles
  static constexpr int PROD = F::kQuant ? (NT == 1 ? 8 : 4) : 0;  // dequantizing warps, half for each tensor
  static constexpr int THREADS = F::kQuant ? 512 : 384;
  static constexpr int PIECES = 4;
  static constexpr int USERS = 4 * NT + 1 + (F::kQuant ? 2 + PROD : 1);  // warps that read a piece
};

template <int D, int FMT>
struct TileShared {
  using C = TileCfg<D, FMT>;
  Work<C::BK, C::ROWS> work;
  Piece piece[C::PIECES];
  uint64_t k_full[C::NS], k_empty[C::NS], v_full[C::NS], v_empty[C::NS];
  uint64_t q_full, q_free, s_full[2], p_full[2], o_done[2], v_land;
  uint64_t raw_full[2][kTileRing], raw_free[2][kTileRing];
  uint64_t piece_full[C::PIECES], piece_free[C::PIECES];
  uint32_t tmem;
  int dead;
};

// A bounded wait that also ends when another role gave up.
template <typename SH>
__device__ __forceinline__ bool tile_wait_warp(SH* sh, const AttnArgs& a, uint64_t* bar, int parity) {
  return warp_wait(smem_u32(bar), parity, &sh->dead, a.pv.err);
}

// Query rows of a piece: row r is token t0 + (rem + r) / rep of the call's rows,
// head of the group (rem + r) % rep.
struct RowMap {
  int t0, rem, rep, head0, p0;
  uint32_t magic;
  __device__ __forceinline__ RowMap(const AttnArgs& a, const Piece& p) {
    const int t = p.r0 / a.rep;
    t0 = p.s.s0 + t;
    p0 = p.s.p0 + t;
    rem = p.r0 - t * a.rep;
    rep = a.rep;
    magic = a.rep_magic;
    head0 = p.head * a.rep;
  }
  __device__ __forceinline__ int token(int r) const { return (int)(((rem + r) * magic) >> 16); }
  __device__ __forceinline__ int position(int r) const { return p0 + token(r); }
  // first element of the row in a tensor with `stride` elements a token
  __device__ __forceinline__ long at(int r, long stride, int D) const {
    const int t = token(r);
    return (long)(t0 + t) * stride + (long)(head0 + rem + r - t * rep) * D;
  }
};

// Blocks [lo, hi) of a piece that a row tile sees any token of.  (One tile: all
// of them, the double-buffered scores count on it.)
template <int D, int FMT>
__device__ __forceinline__ void tile_range(const AttnArgs& a, const Piece& p, int tile, int* lo, int* hi) {
  using C = TileCfg<D, FMT>;
  *lo = 0;
  *hi = p.nblk;
  if (C::NT == 1) return;
  if (tile * 128 >= p.rows) {
    *hi = 0;
    return;
  }
  const RowMap rm(a, p);
  const int first = rm.position(tile * 128), last = rm.position(min(tile * 128 + 127, p.rows - 1));
  *hi = min(max((last < 0 ? 0 : last / C::BK + 1) - p.blk, 0), p.nblk);
  if (a.window > 0) *lo = min(max((int)(max((long)first - a.window + 1, 0L) / C::BK) - p.blk, 0), *hi);
}

// ------------------------------------------------------------------ loader --

template <int D, int FMT>
__device__ __forceinline__ void tile_loader(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int lane) {
  using C = TileCfg<D, FMT>;
  constexpr int CB = D / 64;
  long c = 0;  // blocks so far
  bool ok = true;
  int land = 0;
  for (int k = 0; ok; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) break;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) break;
    const PageRun run(a.pv, p.head);
    for (int j = 0; j < p.nblk; ++j, ++c) {
      const int st = (int)(c % C::NS), par = (int)((c / C::NS) & 1);
      const int tok0 = (p.blk + j) * C::BK;
      const int nt = max(min((p.s.len - tok0 + 15) >> 4, 8), 0);  // records with a token of the sequence
      // lane -> (record, block of 64 columns); head_dim 64 uses 8 lanes, 128 16, 256 all
      const int rec = lane / CB, cb = lane % CB;
      const char* src = nullptr;
      if (rec < nt) {
        const int tok = tok0 + 16 * rec;
        src = run.at(a, page_index(a, p.b, tok), tok) + cb * 2048;
      }
      const uint32_t dst = cb * (C::BK * 128) + rec * 2048;
      ok = tile_wait_warp(sh, a, &sh->k_empty[st], par ^ 1);
      if (!ok) break;
      const uint32_t kb = smem_u32(&sh->k_full[st]);
      if (lane == 0) mbar_expect(kb, nt * CB * 2048);
      __syncwarp();
      if (src) bulk_load(smem + C::K_OFF + st * C::TILE + dst, src, 2048, kb);
      ok = tile_wait_warp(sh, a, &sh->v_empty[st], par ^ 1);
      if (!ok) break;
      const uint32_t vt = smem + C::V_OFF + st * C::TILE, vb = smem_u32(&sh->v_full[st]);
      if (tok0 + C::BK <= p.s.len) {
        if (lane == 0) mbar_expect(vb, nt * CB * 2048);
        __syncwarp();
        if (src) bulk_load(vt + dst, src + a.pv.L.v_off, 2048, vb);
      } else {
        // the sequence ends in this block: the rows behind it are cleared (their weights are zero, their contents anything)
        const uint32_t lb = smem_u32(&sh->v_land);
        if (lane == 0) mbar_expect(lb, nt * CB * 2048);
        __syncwarp();
        if (src) bulk_load(vt + dst, src + a.pv.L.v_off, 2048, lb);
        ok = tile_wait_warp(sh, a, &sh->v_land, land & 1);
        ++land;
        if (!ok) break;
        const int n = max(p.s.len - tok0, 0);
        for (int i = lane; i < (C::BK - n) * (D / 8); i += 32) {
          const int r = n + i / (D / 8), ch = i % (D / 8);
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(vt + (ch >> 3) * (C::BK * 128) + r * 128 + ((ch & 7) << 4)),
                       "r"(0)
                       : "memory");
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(vb);
      }
    }
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}

// ------------------------------------------------------------- dequantizer --

// Brings the records of one tensor (codes and metadata are neighbours) into a
// ring of raw records, ahead of the warps that turn them.
template <int D, int FMT, int VALUE>
__device__ __forceinline__ void raw_loader(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int lane) {
  using C = TileCfg<D, FMT>;
  const PagesLayout& L = a.pv.L;
  const int from = VALUE ? L.v_off : 0, bytes = VALUE ? L.tile_bytes - L.v_off : L.v_off;
  const uint32_t ring = smem + C::RAW_OFF + (VALUE ? a.ring * L.v_off : 0);
  int r = 0, par = 0;
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) return;
    const PageRun run(a.pv, p.head);
    const int end = min((p.blk + p.nblk) * C::BK, p.s.len);
    // 32 records' pages at a time
    for (int tok0 = p.blk * C::BK; tok0 < end; tok0 += 16 * 32) {
      const int mine = tok0 + 16 * lane;
      const int page = mine < end ? page_index(a, p.b, mine) : 0;
      for (int i = 0; i < 32 && tok0 + 16 * i < end; ++i) {
        const int pg = __shfl_sync(0xffffffffu, page, i);
        if (!tile_wait_warp(sh, a, &sh->raw_free[VALUE][r], par ^ 1)) return;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sh->raw_full[VALUE][r]);
          mbar_expect(bar, bytes);
          bulk_load(ring + r * bytes, run.at(a, pg, tok0 + 16 * i) + from, bytes, bar);
        }
        if (++r == a.ring) r = 0, par ^= 1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}

// Keys (VALUE 0) or values (1) of all pieces: a thread turns a run of 32 channels
// of one token into four 16-byte chunks of the operand tile; tid: thread among
// those of the tensor.  The loop body is kept small: with the many roles of this
// kernel, unrolled over a block it ran out of the instruction cache.
template <int D, int FMT, int VALUE>
__device__ __forceinline__ void tile_dequantizer(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int tid) {
  using C = TileCfg<D, FMT>;
  using F = typename C::F;
  constexpr int BITS = F::KB == 16 ? 4 : (VALUE ? F::VB : F::KB);
  constexpr int THREADS = 16 * C::PROD, PPT = D / 32;
  constexpr int RECS = THREADS / (16 * PPT);  // records turned at once
  static_assert(RECS >= 1 && RECS <= 2, "the ring holds two records at least");
  constexpr int WC = BITS / 4;                // words of a chunk of 8 channels
  const int lane = tid & 31, piece = tid % PPT, rec = tid / (16 * PPT), row = (tid / PPT) & 15;
  const PagesLayout& L = a.pv.L;
  const int meta = VALUE ? L.vm_off - L.v_off : L.km_off, lg = VALUE ? L.v_lg : L.k_lg;
  const uint32_t raw = smem + C::RAW_OFF + (VALUE ? a.ring * L.v_off : 0);
  const int raw_bytes = VALUE ? L.tile_bytes - L.v_off : L.v_off;
  const uint32_t codes_at = row * (D * BITS / 8) + piece * (4 * BITS);
  const uint32_t meta_at = meta + (row * (D >> lg) + ((piece * 32) >> lg)) * 4;
  // lanes of other column blocks store their four chunks in another order, so
  // that the 8 lanes of a phase touch 8 different groups of banks
  const int turn = D == 64 ? 0 : (D == 128 ? 2 * (piece >> 1) : piece >> 1);
  int st = 0, par = 0, r = 0, rpar = 0;
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) return;
    int tok = p.blk * C::BK;
    // A unit's codes and metadata.  Every record with a token of the sequence
    // arrives; rows behind its end become zero (zero + code * step = 0), whatever
    // the page holds there.
    auto take = [&](int tok, uint32_t* w, uint32_t* zs) -> bool {
#pragma unroll
      for (int i = 0; i < 4 * WC; ++i) w[i] = 0;
      *zs = 0;
      int rr = r, pp = rpar;
#pragma unroll
      for (int i = 0; i < RECS; ++i) {
        if (tok + 16 * i >= p.s.len) continue;
        if (!tile_wait_warp(sh, a, &sh->raw_full[VALUE][rr], pp)) return false;
        if (RECS == 1 || rec == i) {
          const uint32_t from = raw + rr * raw_bytes;
          ldsv<4 * WC>(from + codes_at, w);
          *zs = lds32(from + meta_at);
        }
        if (++rr == a.ring) rr = 0, pp ^= 1;
      }
      return true;
    };
    // Its records go back: the fence orders each lane's loads before the bulk copies
    // into the same bytes, which go another way (without it a copy overtook loads that
    // waited behind the matrix operands), the warp's barrier the lanes before the
    // arrival.  (The records held until their values are stored: 703 us against 579
    // for 2 x 600 tokens at 20000, 16 over 2 heads of 256, 8 bits.)
    auto give_back = [&](int tok) {
      fence_async();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < RECS; ++i)
        if (tok + 16 * i < p.s.len) {
          if (lane == 0) mbar_arrive(smem_u32(&sh->raw_free[VALUE][r]));
          if (++r == a.ring) r = 0, rpar ^= 1;
        }
    };
    auto turn_unit = [&](int tok, uint32_t* w, uint32_t zs, uint32_t out) {
      if (tok + rec * 16 + row >= p.s.len) zs = 0;
      const __half2 z = __low2half2(as_h2(zs)), s = __high2half2(as_h2(zs));
#pragma unroll
      for (int b = 1; b < 4; b <<= 1)  // the words of chunk k to place k ^ turn
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(c & b))
#pragma unroll
            for (int e = 0; e < WC; ++e) {
              const uint32_t x = w[WC * c + e], y = w[WC * (c ^ b) + e];
              w[WC * c + e] = (turn & b) ? y : x;
              w[WC * (c ^ b) + e] = (turn & b) ? x : y;
            }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[4];
        if constexpr (BITS == 8) {
          y[0] = bytes<0>(w[2 * c], s, z);
          y[1] = bytes<1>(w[2 * c], s, z);
          y[2] = bytes<0>(w[2 * c + 1], s, z);
          y[3] = bytes<1>(w[2 * c + 1], s, z);
        } else {
          y[0] = nibbles<0>(w[c], s, z);
          y[1] = nibbles<1>(w[c], s, z);
          y[2] = nibbles<2>(w[c], s, z);
          y[3] = nibbles<3>(w[c], s, z);
        }
        const int at = (4 * (piece & 1) + (c ^ turn)) ^ (row & 7);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(out + (at << 4)), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                     : "memory");
      }
    };
#pragma unroll 1
    for (int j = 0; j < p.nblk; ++j) {
      if (!tile_wait_warp(sh, a, VALUE ? &sh->v_empty[st] : &sh->k_empty[st], par ^ 1)) return;
      uint32_t out = smem + (VALUE ? C::V_OFF : C::K_OFF) + st * C::TILE + (piece >> 1) * (128 * 128) + (rec * 16 + row) * 128;
      constexpr int UT = 16 * RECS;  // tokens of a unit; two units a turn, for the latencies of one to hide the other's
#pragma unroll 1
      for (int u = 0; u < C::BK; u += 2 * UT, tok += 2 * UT, out += 2 * UT * 128) {
        uint32_t w0[4 * WC], w1[4 * WC], z0, z1;
        if (!take(tok, w0, &z0)) return;
        give_back(tok);
        if (!take(tok + UT, w1, &z1)) return;
        give_back(tok + UT);
        turn_unit(tok, w0, z0, out);
        turn_unit(tok + UT, w1, z1, out + UT * 128);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(VALUE ? &sh->v_full[st] : &sh->k_full[st]));
      if (++st == C::NS) st = 0, par ^= 1;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}

// -------------------------------------------------------------- matrix unit --

// The whole warp follows the barriers; one elected lane issues.
template <int D, int FMT>
__device__ __forceinline__ void tile_mma(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem) {
  using C = TileCfg<D, FMT>;
  constexpr uint32_t S_DESC = mma_desc(128, C::BK, C::F::kBf16, false);
  constexpr uint32_t O_DESC = mma_desc(128, D, C::F::kBf16, true);
  const uint32_t tm = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const uint64_t q0 = smem_desc(smem + C::Q_OFF, 16, 1024), k0 = smem_desc(smem + C::K_OFF, 16, 1024);
  const uint64_t v0 = smem_desc(smem + C::V_OFF, C::BK * 128, 1024);
  int ks = 0, kpar = 0, vs = 0, vpar = 0;  // stage to read next, its phase
  int bc = 0;                              // score buffers handed out (one tile)
  int pc[2] = {0, 0};
  // S of a tile with the keys of stage ks; O of a tile with the values of stage vs.
  // (Scoring the next block's first 64 keys into the columns that the weights leave
  // free, ahead of the value product, was slower: 995 us against 820 for a chunk of
  // 2048 at 32k tokens; products of 64 columns wait for shared memory.)
  auto scores = [&](int buf, int tile) {
    const uint64_t q = q0 + (uint64_t)(tile * (C::TILE >> 4)), k = k0 + (uint64_t)(ks * (C::TILE >> 4));
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint64_t at = ((i >> 2) * (128 * 128) + (i & 3) * 32) >> 4;
        mma_ss(tm + buf * 128, q + at, k + at, S_DESC, i > 0);
      }
      mma_commit(smem_u32(&sh->s_full[buf]));
    }
    __syncwarp();
  };
  auto values = [&](int buf, int tile, int add) {
    const uint64_t v = v0 + (uint64_t)(vs * (C::TILE >> 4));
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < C::BK / 16; ++i)
        mma_ts(tm + 256 + tile * D, tm + buf * 128 + i * 8, v + (uint64_t)(i * 2048 >> 4), O_DESC, i > 0 ? 1 : add);
      mma_commit(smem_u32(&sh->o_done[tile]));
    }
    __syncwarp();
  };
  // the stages go back when what was issued so far is done
  auto free_k = [&](bool queries_too) {
    if (elect_one()) {
      mma_commit(smem_u32(&sh->k_empty[ks]));
      if (queries_too) mma_commit(smem_u32(&sh->q_free));
    }
    __syncwarp();
    if (++ks == C::NS) ks = 0, kpar ^= 1;
  };
  auto free_v = [&]() {
    if (elect_one()) mma_commit(smem_u32(&sh->v_empty[vs]));
    __syncwarp();
    if (++vs == C::NS) vs = 0, vpar ^= 1;
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const int n = __shfl_sync(0xffffffffu, sh->piece[slot].nblk, 0);
    if (n == 0) return;
    if (!tile_wait_warp(sh, a, &sh->q_full, k & 1)) return;
    if (!tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
    tc_after_sync();
    if (C::NT == 2) {
      int lo[2], hi[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tile_range<D, FMT>(a, sh->piece[slot], i, &lo[i], &hi[i]);
        lo[i] = __shfl_sync(0xffffffffu, lo[i], 0);
        hi[i] = __shfl_sync(0xffffffffu, hi[i], 0);
      }
      auto sees = [&](int i, int j) { return j >= lo[i] && j < hi[i]; };
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (sees(i, 0)) scores(i, i);
      free_k(n == 1);
      for (int j = 0; j < n; ++j) {
        bool have_k = false;
        if (!tile_wait_warp(sh, a, &sh->v_full[vs], vpar)) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (sees(i, j)) {
            if (!tile_wait_warp(sh, a, &sh->p_full[i], pc[i] & 1)) return;
            ++pc[i];
            tc_after_sync();
            values(i, i, j > lo[i]);
          }
          if (i == 1) free_v();
          if (j + 1 < n && sees(i, j + 1)) {
            if (!have_k && !tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
            have_k = true;
            tc_after_sync();
            scores(i, i);
          }
        }
        if (j + 1 < n) {
          if (!have_k && !tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
          free_k(j + 2 == n);
        }
      }
    } else {
      scores(bc & 1, 0);
      free_k(n == 1);
      for (int j = 0; j < n; ++j) {
        const int buf = bc & 1;
        if (j + 1 < n) {
          if (!tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
          tc_after_sync();
          scores(buf ^ 1, 0);
          free_k(j + 2 == n);
        }
        if (!tile_wait_warp(sh, a, &sh->v_full[vs], vpar)) return;
        if (!tile_wait_warp(sh, a, &sh->p_full[buf], (bc >> 1) & 1)) return;
        tc_after_sync();
        values(buf, 0, j > 0);
        free_v();
        ++bc;
      }
    }
    if (elect_one()) mbar_arrive(smem_u32(&sh->piece_free[slot]));
    __syncwarp();
  }
}

// ------------------------------------------------------------------ softmax --

// A warp's 32 rows of queries into the swizzled operand tile, D / 8 lanes a row
// (zeros behind the item's rows); returns what the lane's row's scores are to be
// multiplied by.  row0: the warp's first row inside the tile.
template <int D, int FMT>
__device__ __forceinline__ float tile_query(const AttnArgs& a, const RowMap& rm, int rows, int tile_row, int row0,
                                            uint32_t tile, int lane) {
  using F = Fmt<FMT>;
  constexpr int LPR = D / 8, RPI = 32 / LPR, U = LPR < 16 ? LPR : 16;  // lanes a row, rows a step, steps in flight
  const int g = lane / LPR, c = lane % LPR;
  float sc = a.scale_log2;
  for (int it0 = 0; it0 < LPR; it0 += U) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = tile_row + row0 + (it0 + u) * RPI + g;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + rm.at(min(r, rows - 1), a.q_stride, D) + c * 8;
      if (a.q_aligned) {
        w[u] = *reinterpret_cast<const uint4*>(src);
      } else {
        uint16_t* e = reinterpret_cast<uint16_t*>(&w[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = src[i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u, row = row0 + it * RPI + g;
      uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      if (F::kQuant && a.q_bf16) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int E = query_exp(mx);
        const float f0 = exp2i(E / 2), f1 = exp2i(E - E / 2);
        const float y = __shfl_sync(0xffffffffu, row_factor(a, E), (lane % RPI) * LPR);
        if (lane / RPI == it) sc = y;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = pack2<false>(__uint_as_float(x[i] << 16) * f0 * f1, __uint_as_float(x[i] & 0xffff0000u) * f0 * f1);
      }
      if (tile_row + row >= rows) x[0] = x[1] = x[2] = x[3] = 0;
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(tile + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)),
                   "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                   : "memory");
    }
  }
  return sc;
}

template <int D, int FMT>
__device__ __forceinline__ void tile_softmax(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int tile, int tid) {
  using C = TileCfg<D, FMT>;
  using F = typename C::F;
  constexpr int BK = C::BK;
  const int lane = tid & 31, row = tid & 127;
  const uint32_t lanes = (uint32_t)((row >> 5) * 32) << 16;
  const uint32_t tm = sh->tmem + lanes, o_col = 256 + tile * D;
  int bc = 0, ob = 0;  // blocks read (of this tile), value products asked for
  int od = 0;          // value products known to be done
  // Waits for the first n products.  Each phase is waited for, in order, and before
  // the next product is asked for: a barrier's parity tells only two phases apart.
  auto products = [&](int n) {
    for (; od < n; ++od)
      if (!tile_wait_warp(sh, a, &sh->o_done[tile], od & 1)) return false;
    tc_after_sync();
    return true;
  };
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) return;
    if (k > 0 && !tile_wait_warp(sh, a, &sh->q_free, (k - 1) & 1)) return;
    const int r = tile * 128 + row;
    const RowMap rm(a, p);
    const uint32_t q_tile = smem + C::Q_OFF + tile * C::TILE;
    float sc = a.scale_log2;
    if (tile * 128 < p.rows) sc = tile_query<D, FMT>(a, rm, p.rows, tile * 128, row & ~31, q_tile, lane);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->q_full));
    if (tile * 128 < p.rows) {
      const int pos = rm.position(min(r, p.rows - 1));
      // the tile's first and last position: blocks between need no mask
      const int pos_lo = rm.position(tile * 128), pos_hi = rm.position(min(tile * 128 + 127, p.rows - 1));
      int j0, j1;
      tile_range<D, FMT>(a, p, tile, &j0, &j1);
      float m = -INFINITY;
      float2 l = make_float2(0.0f, 0.0f);
      for (int j = j0; j < j1; ++j, ++bc, ++ob) {
        const int buf = C::NT == 2 ? tile : (bc & 1);
        if (!tile_wait_warp(sh, a, &sh->s_full[buf], C::NT == 2 ? bc & 1 : (bc >> 1) & 1)) return;
        tc_after_sync();
        const uint32_t sb = tm + buf * 128;
        const int tok0 = (p.blk + j) * BK;
        const bool edge = tok0 + BK - 1 > pos_lo || (a.window > 0 && tok0 <= pos_hi - a.window);
        const int hi = pos - tok0, lo = a.window > 0 ? pos - a.window - tok0 : -1;  // visible columns: lo < c <= hi
        auto hide = [&](uint32_t* e, int q) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (q * 32 + c > hi || q * 32 + c <= lo) e[c] = 0xff800000u;
        };
        uint32_t s[64], w[64];
        float2 add;
        // Most blocks leave the running maximum alone, so the weights are taken under
        // it while the block's maximum is found.  Where that passes it by 2^8, and in
        // an item's first block, the row is read once more for its maximum.
        bool find_max = j == j0;
        for (;;) {
          if (find_max) {
            float top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < BK / 32; ++q) {
              tmem_ld32(sb + q * 32, s);
              if (edge) hide(s, q);
#pragma unroll
              for (int c = 0; c < 32; c += 2) top = fmaxf(fmaxf(top, __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
            }
            const float to = fmaxf(m, top * sc);
            if (j > j0) {
              const float f = to == -INFINITY ? 1.0f : fast_exp2(m - to);
              if (!products(ob)) return;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                tmem_ld32(tm + o_col + c, s);
#pragma unroll
                for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * f);
                tmem_st32(tm + o_col + c, s);
              }
              l.x *= f;
              l.y *= f;
            }
            m = to;
          }
          const float base = m == -INFINITY ? 0.0f : 7.0f - m;
          const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(base, base);
          add = make_float2(0.0f, 0.0f);
          float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
          for (int q = 0; q < BK / 32; ++q) {
            if (q % 2 == 0) tmem_ld64(sb + q * 32, s);
            uint32_t* e = s + q % 2 * 32;
            if (edge) hide(e, q);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float2 x = make_float2(__uint_as_float(e[c]), __uint_as_float(e[c + 1]));
              if (c & 2) x1 = fmaxf(fmaxf(x1, x.x), x.y);
              else x0 = fmaxf(fmaxf(x0, x.x), x.y);
              x = fma2(x, sc2, nb2);
              x.x = fast_exp2(x.x);
              x.y = fast_exp2(x.y);
              add = add2(add, x);
              w[q * 16 + c / 2] = pack2<F::kBf16>(x.x, x.y);
            }
          }
          const bool over = fmaxf(x0, x1) * sc > m + 8.0f;
          if (find_max || !__any_sync(0xffffffffu, over)) break;
          find_max = true;
        }
        l = add2(l, add);
        if (C::NT == 2) od = ob;  // (two tiles: these scores came after the last product)
        else if (!products(ob)) return;
        tmem_st32(sb, w);
        tmem_st32(sb + 32, w + 32);
        tmem_wait_st();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[buf]));
      }
      // ---- the item's output, or this CTA's part of it
      if (!products(ob)) return;
      const float sum = l.x + l.y;
      const bool whole = p.has_first && p.has_last, has = r < p.rows;
      const float f = whole ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
      const long slot_row = ((long)blockIdx.x * 2 + (p.has_first ? 1 : 0)) * C::ROWS + r;
      // Whole rows go through the query tile's place (its last product is done),
      // so that the stores are D / 8 lanes a row.
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(tm + o_col + c, o);
        if (j1 == j0) {  // no block: O was never written
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = __uint_as_float(o[e + 2 * i]) * f, v = __uint_as_float(o[e + 2 * i + 1]) * f;
              x[i] = a.q_bf16 ? pack2<true>(u, v) : pack2<false>(u, v);
            }
            const int ch = (c + e) / 8;
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(q_tile + (ch >> 3) * (128 * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4)),
                         "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
        } else if (has) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(a.part_o + slot_row * D + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (whole) {
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const int g = lane / LPR, ch = lane % LPR;
        __syncwarp();
#pragma unroll 4
        for (int it = 0; it < LPR; ++it) {
          const int rw = (row & ~31) + it * RPI + g;
          uint4 w;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(q_tile + (ch >> 3) * (128 * 128) + rw * 128 + (((ch & 7) ^ (rw & 7)) << 4))
                       : "memory");
          if (tile * 128 + rw < p.rows)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + rm.at(tile * 128 + rw, (long)a.q_heads * D, D) + ch * 8) = w;
        }
        __syncwarp();
      }
      if (!whole && has) *reinterpret_cast<float2*>(a.part_ml + slot_row * 2) = make_float2(m, sum);
      tc_before_sync();
    }
    if (tile == 0 && row == 0 && p.has_first && !p.has_last) {
      SplitHead h = {};
      h.parts = cta_of(&sh->work, p.item1 - 1) - (int)blockIdx.x + 1;
      h.rows = p.rows, h.row0 = p.r0, h.q_row = p.s.s0, h.head = p.head;
      a.split[blockIdx.x] = h;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}

// ------------------------------------------------------------------- kernel --

template <int D, int FMT>
__global__ void __launch_bounds__(TileCfg<D, FMT>::THREADS, 1) pages_tile_kernel(const __grid_constant__ AttnArgs a) {
  using C = TileCfg<D, FMT>;
  using F = typename C::F;
  extern __shared__ char raw[];
  __shared__ TileShared<D, FMT> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), F::kQuant ? C::PROD / 2 : 1);
      mbar_init(smem_u32(&sh.v_full[i]), F::kQuant ? C::PROD / 2 : 1);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.o_done[i]), 1);
    }
    mbar_init(smem_u32(&sh.q_full), 4 * C::NT);
    mbar_init(smem_u32(&sh.q_free), 1);
    mbar_init(smem_u32(&sh.v_land), 1);
    for (int i = 0; i < C::PIECES; ++i) {
      mbar_init(smem_u32(&sh.piece_full[i]), 1);
      mbar_init(smem_u32(&sh.piece_free[i]), C::USERS);
    }
    for (int i = 0; i < kTileRing; ++i)
      for (int t = 0; t < 2; ++t) {
        mbar_init(smem_u32(&sh.raw_full[t][i]), 1);
        mbar_init(smem_u32(&sh.raw_free[t][i]), F::kQuant ? C::PROD / 2 : 1);
      }
    sh.dead = 0;
    fence_mbar_init();
  }
  pdl_wait();
  plan_work<C::BK, C::ROWS, false>(a, &sh.work, reinterpret_cast<long*>(raw + C::SMEM + a.ring * a.pv.L.tile_bytes));  // (its barriers also publish the initialisation above)
  pdl_trigger();
  if (threadIdx.x == 0) a.split[blockIdx.x].parts = 0;
  if ((int)blockIdx.x >= sh.work.ctas) return;
  if (warp == 8) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();

  // Registers over codes: 512 threads start with 128 each (65536); two tiles take
  // 256 * 176 + 128 * 72 + 128 * 88 = 65536 of them, one tile 128 * 176 +
  // 128 * 72 + 256 * 88 = 54272.
  if (warp < 4 * C::NT) {
    if constexpr (F::kQuant) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
    tile_softmax<D, FMT>(a, &sh, smem, warp >> 2, threadIdx.x);
  } else if (warp < 8) {
    if constexpr (F::kQuant) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
      tile_dequantizer<D, FMT, 1>(a, &sh, smem, threadIdx.x - 128);  // (one tile) values
    }
  } else if (warp < 12) {
    if constexpr (F::kQuant) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp == 8) {
      tile_mma<D, FMT>(a, &sh, smem);
    } else if (warp == 9) {
      if constexpr (F::kQuant) raw_loader<D, FMT, 0>(a, &sh, smem, lane);
      else tile_loader<D, FMT>(a, &sh, smem, lane);
    } else if (warp == 10) {
      // the pieces of this CTA's units, ahead of the others; nblk 0 ends
      long u = cta_begin(&sh.work, blockIdx.x);
      const long end = cta_begin(&sh.work, blockIdx.x + 1);
      for (int k = 0;; ++k) {
        const int slot = k % C::PIECES;
        if (k >= C::PIECES && !tile_wait_warp(&sh, a, &sh.piece_free[slot], (k / C::PIECES - 1) & 1)) break;
        Piece p = {};
        if (u < end) {
          p = find_piece(a, &sh.work, u, end);
          // its queries to the L2 cache, while the piece before is worked on
          const RowMap rm(a, p);
          for (int r = lane; r < p.rows; r += 32) {
            const char* row = static_cast<const char*>(a.q) + rm.at(r, a.q_stride, D) * 2;
#pragma unroll
            for (int c = 0; c < D * 2; c += 128) prefetch_l2(row + c);
          }
        }
        u += p.nblk;
        if (lane == 0) {
          sh.piece[slot] = p;
          mbar_arrive(smem_u32(&sh.piece_full[slot]));
        }
        __syncwarp();
        if (p.nblk == 0) break;
      }
    } else {
      if constexpr (F::kQuant) raw_loader<D, FMT, 1>(a, &sh, smem, lane);
    }
  } else {
    if constexpr (F::kQuant) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
      if (C::NT == 1 || warp < 14) tile_dequantizer<D, FMT, 0>(a, &sh, smem, threadIdx.x - 384);
      else tile_dequantizer<D, FMT, 1>(a, &sh, smem, threadIdx.x - 448);
    }
  }
  __syncwarp();
  if (*(volatile int*)&sh.dead) {  // given up: what is in flight lands before memory is given back
    const unsigned long long t0 = time_ns();
    while (time_ns() - t0 < 5000000ull) __nanosleep(1000);
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 8) tmem_free(sh.tmem, 512);
}

template <int D>
AttnKernel tile_kernel_dim(int fmt) {
  switch (fmt) {
#define KVQ_TILE(f) \
  case f: return {(const void*)pages_tile_kernel<D, f>, (size_t)TileCfg<D, f>::SMEM, TileCfg<D, f>::THREADS, 0, 0};
    KVQ_TILE(kFmtF16)
    KVQ_TILE(kFmtBf16)
    KVQ_TILE(kFmt88)
    KVQ_TILE(kFmt44)
    KVQ_TILE(kFmt84)
    KVQ_TILE(kFmt48)
#undef KVQ_TILE
  }
  return {};
}

}  // namespace kvq
