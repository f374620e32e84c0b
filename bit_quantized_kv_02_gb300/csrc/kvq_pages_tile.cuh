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
//  - dequantizers (codes): three warps per tensor (four with one row tile) copy records
//    ahead and turn their codes into fp16 operand tiles (the value the page stands for,
//    one rounding);
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
// Measured: 2048 new tokens at 30720, 32 query heads over 8 of 128, bf16 pages: 790 us,
// 1.35 PFLOP/s (71 % of a large library product).  A CTA takes 418 blocks of two tiles, so
// a block takes 1.89 us, of which its products would take 1.34 at the library product's
// rate: a tile's chain of scores, softmax, value product and the signals between them is
// what is left.  509 tokens at 130563, 16 query heads over 2 of 256, 4-bit keys and 8-bit
// values: 1261 us, 0.87 PFLOP/s: the dequantizers' traffic in shared memory slows the
// products (each CTA turns every code for 128 rows), and keys come as two products of 64
// columns.  Prompts of up to 2048 tokens, 40 heads of 128, window 1024: 335 us.  A CTA has
// 68 blocks there, in 10.5 pieces, which would take 128 us at the chunk's pace; the rest
// (queries and outputs that no other piece covers, blocks with a mask, a second read of
// the scores in each piece's first block) was not measured apart.
// Masked: 16 sequences with trees of 64 tokens over 1k to 16k bf16 tokens, 32 over 8 heads
// of 128, 186 us (floor 105, bytes and products near each other); 125 drafted tokens at
// 130900, 16 over 2 heads of 256, 4 and 8 bits, 342 us (floor 141, products); 8 decoder
// prompts of up to 448 tokens over 8190 8-bit tokens, 326 us (floor 83, products).
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
  // Where only one stage fits it is handed over by halves: the next block's first half is
  // made while the products take the second.
  static constexpr int PT = D == 256 ? 64 : 128;   // tokens of a part of a stage
  static constexpr int SP = NS * (BK / PT);        // parts of the stages
  static constexpr int TILE = 128 * D * 2;         // bytes of a Q, K or V tile
  static constexpr int Q_OFF = 0, K_OFF = NT * TILE, V_OFF = K_OFF + NS * TILE;
  // over codes, what the dequantizing warps copied ahead comes behind the tiles, as many
  // units a warp (a.ring) as the 227 KB of a CTA allow
  static constexpr int TURN = D == 64 ? 1 : 2;  // runs (32 lanes x 32 channels) of a unit
  static constexpr __host__ __device__ int unit_bytes(int bits) { return TURN * 32 * (4 * bits + 4); }
  static constexpr int RAW_OFF = V_OFF + NS * TILE;
  static constexpr int SMEM = RAW_OFF + 1024;  // + alignment of the tiles
  static constexpr int PROD = F::kQuant ? (NT == 1 ? 8 : 6) : 0;  // dequantizing warps, half for each tensor
  static constexpr int THREADS = F::kQuant ? 512 : 384;
  static constexpr int PIECES = 4;
  static constexpr int COPIES = F::kQuant ? PROD / 2 * (unit_bytes(F::KB) + unit_bytes(F::VB)) : 0;  // bytes of a unit of every warp
  static constexpr int USERS = 4 * NT + 1 + (F::kQuant ? PROD : 1);  // warps that read a piece
};

template <int D, int FMT>
struct TileShared {
  using C = TileCfg<D, FMT>;
  Work<C::BK, C::ROWS> work;
  Piece piece[C::PIECES];
  uint64_t k_full[C::SP], k_empty[C::SP], v_full[C::SP], v_empty[C::SP];
  uint64_t q_full, q_free, s_full[2], p_full[2], o_done[2], v_land;
  uint64_t piece_full[C::PIECES], piece_free[C::PIECES];
  uint64_t met[4];         // warps of both tiles that hold the same rows
  float2 stats[2][C::NT == 2 ? 128 : 1];  // maxima and sums that they exchange
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

// Do the two row tiles share a piece's blocks between them, both holding its rows?  One
// tile alone leaves the tensor cores to wait for its softmax: 8 trees of 64 tokens over
// 8192, 16-bit pages, 12 heads of 64 88 -> 59 us, 16 tokens, 32 over 8 heads of 128 72 ->
// 66.  Over codes the dequantizing warps bound both forms (71 us and 68).  (Masked kernels
// only: the causal ones keep their order of sums.)
template <int D, int FMT, bool MASK>
__device__ __forceinline__ bool shared_rows(int rows) {
  return MASK && TileCfg<D, FMT>::NT == 2 && !Fmt<FMT>::kQuant && rows <= 128;
}

// Blocks [lo, hi) of a piece that a row tile sees any token of.  (One tile: all
// of them, the double-buffered scores count on it.  MASK: all of them too, the rows
// see past and new tokens alike.)
template <int D, int FMT, bool MASK>
__device__ __forceinline__ void tile_range(const AttnArgs& a, const Piece& p, int tile, int* lo, int* hi) {
  using C = TileCfg<D, FMT>;
  *lo = 0;
  *hi = p.nblk;
  if (C::NT == 1) return;
  if (tile * 128 >= p.rows) {
    *hi = 0;
    return;
  }
  if (MASK) return;
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
  constexpr int HALVES = C::BK / C::PT;
  int st = 0, par = 0;  // first part of the block's stage, its phase
  int land = 0;
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) return;
    const PageRun run(a.pv, p.head);
    for (int j = 0; j < p.nblk; ++j) {
      // lane -> (record, block of 64 columns); head_dim 64 uses 8 lanes, 128 16, 256 all
      const int rec = lane / CB, cb = lane % CB, blk0 = (p.blk + j) * C::BK;
      const char* src = nullptr;
      if (rec < C::BK / 16 && blk0 + 16 * rec < p.s.len) {
        const int tok = blk0 + 16 * rec;
        src = run.at(a, page_index(a, p.b, tok), tok) + cb * 2048;
      }
      const uint32_t stage = smem + st / HALVES * C::TILE, dst = cb * (C::BK * 128) + rec * 2048;
      // Keys, all parts of the block, before values: the products of the next block's
      // scores come before those of this one's values.
      for (int h = 0; h < HALVES; ++h) {
        const int tok0 = blk0 + h * C::PT, nt = max(min((p.s.len - tok0 + 15) >> 4, C::PT / 16), 0);  // records with a token of the sequence
        const bool mine = src && (HALVES == 1 || rec / (C::PT / 16) == h);
        if (!tile_wait_warp(sh, a, &sh->k_empty[st + h], par ^ 1)) return;
        const uint32_t kb = smem_u32(&sh->k_full[st + h]);
        if (lane == 0) mbar_expect(kb, nt * CB * 2048);
        __syncwarp();
        if (mine) bulk_load(stage + C::K_OFF + dst, src, 2048, kb);
      }
      for (int h = 0; h < HALVES; ++h) {
        const int tok0 = blk0 + h * C::PT, nt = max(min((p.s.len - tok0 + 15) >> 4, C::PT / 16), 0);
        const bool mine = src && (HALVES == 1 || rec / (C::PT / 16) == h);
        if (!tile_wait_warp(sh, a, &sh->v_empty[st + h], par ^ 1)) return;
        const uint32_t vt = stage + C::V_OFF, vb = smem_u32(&sh->v_full[st + h]);
        if (tok0 + C::PT <= p.s.len) {
          if (lane == 0) mbar_expect(vb, nt * CB * 2048);
          __syncwarp();
          if (mine) bulk_load(vt + dst, src + a.pv.L.v_off, 2048, vb);
        } else {
          // the sequence ends in this part: the rows behind it are cleared (their weights are zero, their contents anything)
          const uint32_t lb = smem_u32(&sh->v_land);
          if (lane == 0) mbar_expect(lb, nt * CB * 2048);
          __syncwarp();
          if (mine) bulk_load(vt + dst, src + a.pv.L.v_off, 2048, lb);
          if (!tile_wait_warp(sh, a, &sh->v_land, land & 1)) return;
          ++land;
          const int n = max(p.s.len - tok0, 0);
          for (int i = lane; i < (C::PT - n) * (D / 8); i += 32) {
            const int r = h * C::PT + n + i / (D / 8), ch = i % (D / 8);
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};\n" ::"r"(vt + (ch >> 3) * (C::BK * 128) + r * 128 + ((ch & 7) << 4)),
                         "r"(0)
                         : "memory");
          }
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(vb);
        }
      }
      if ((st += HALVES) == C::SP) st = 0, par ^= 1;
    }
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}

// ------------------------------------------------------------- dequantizer --

// Codes of keys (value 0) or values (1) of all pieces into operand tiles.  A warp turns
// whole records, every WARPS-th; a lane turns runs of 32 channels of one token into four
// 16-byte chunks of the tile.  What a lane turns it copies itself, some units (one or two
// runs and their metadata) ahead, into places in shared memory that no other lane reads:
// its copies ask for no barrier and no fence, and it waits for its own oldest one alone.
// (Records brought by bulk copies into a ring that two loader warps filled: 125 drafted
// tokens at 130900, 16 over 2 heads of 256, 372 us; a record's place, given back and
// filled again, cost more than turning it.)  Keys and values share the code where their
// bits do, and a turn is one unit: with the many roles of this kernel its hot code is
// what the instruction cache holds.  warp: among those of the tensor.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// All of this thread's groups but the last n (0 .. 3) have landed.
__device__ __forceinline__ void copy_wait(int n) {
  if (n == 3) asm volatile("cp.async.wait_group 3;\n" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;\n" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
  else asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

template <int D, int FMT, int BITS>
__device__ __forceinline__ void tile_dequantizer(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int value, int warp, int lane) {
  using C = TileCfg<D, FMT>;
  constexpr int WARPS = C::PROD / 2, PPT = D / 32, ROWS = 32 / PPT;  // rows of a run of the warp
  constexpr int RUNS = 16 / ROWS, TURN = C::TURN;                    // runs of a record, of a unit
  constexpr int WC = BITS / 4;                                       // words of a chunk of 8 channels
  constexpr int UNITS = RUNS / TURN, PER = C::PT / 16;               // units of a record, records of a part
  static_assert(WARPS <= PER, "each warp has a record of each part");
  const int piece = lane % PPT, row = lane / PPT;
  const PagesLayout& L = a.pv.L;
  const int lg = value ? L.v_lg : L.k_lg, meta_run = ROWS * (D >> lg) * 4;
  const int codes_at = (value ? L.v_off : 0) + row * (D * BITS / 8) + piece * (4 * BITS);
  const int meta_at = (value ? L.vm_off : L.km_off) + (row * (D >> lg) + ((piece * 32) >> lg)) * 4;
  uint64_t* const empty = value ? sh->v_empty : sh->k_empty;
  uint64_t* const ready = value ? sh->v_full : sh->k_full;
  const uint32_t tiles = smem + (value ? C::V_OFF : C::K_OFF) + (piece >> 1) * (128 * 128);
  // the lane's places: [unit in flight][run][16 bytes, WC of them], then the metadata
  constexpr int UNIT = C::unit_bytes(BITS);
  const uint32_t mine = smem + C::RAW_OFF + (value ? WARPS * a.ring * C::unit_bytes(C::F::KB) : 0) + warp * a.ring * UNIT;
  const uint32_t my_codes = mine + lane * 16, my_meta = mine + TURN * WC * 512 + lane * 4;
  // lanes of other column blocks store their four chunks in another order, so
  // that the 8 lanes of a phase touch 8 different groups of banks
  const int turn = D == 64 ? 0 : (D == 128 ? 2 * (piece >> 1) : piece >> 1);
  int st = 0, par = 0;
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const Piece p = sh->piece[slot];
    if (p.nblk == 0) return;
    const PageRun run(a.pv, p.head);
    const int all = (p.nblk * (C::BK / 16) - warp + WARPS - 1) / WARPS * UNITS;  // the warp's units
    // Unit u is part u % UNITS of the warp's record u / UNITS, 16 * WARPS tokens from the
    // one before.  A record's page is read while the one before is copied.
    int tok = p.blk * C::BK + warp * 16, part = 0, put = 0;  // of the next unit to be copied; its place
    const int end = min((p.blk + p.nblk) * C::BK, p.s.len);
    int page = tok < end ? page_index(a, p.b, tok) : 0;
    const char* src = nullptr;
    auto bring = [&]() {
      if (tok < end) {
        if (part == 0) {
          src = run.at(a, page, tok);
          if (tok + 16 * WARPS < end) page = page_index(a, p.b, tok + 16 * WARPS);
        }
        const uint32_t to = put * UNIT;
        const char* codes = src + codes_at + part * (TURN * ROWS * D * BITS / 8);
        const char* meta = src + meta_at + part * TURN * meta_run;
#pragma unroll
        for (int y = 0; y < TURN; ++y) {
#pragma unroll
          for (int e = 0; e < WC; ++e) copy_async16(my_codes + to + (y * WC + e) * 512, codes + y * (ROWS * D * BITS / 8) + e * 16);
          copy_async4(my_meta + to + y * 128, meta + y * meta_run);
        }
      }
      copy_commit();  // (a group a unit, empty ones included)
      if (++part == UNITS) part = 0, tok += 16 * WARPS;
      if (++put == a.ring) put = 0;
    };
    int get = 0, now = 0;  // place of the next unit to be turned; the part that is being made
    auto part_done = [&]() {
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ready[st]));
      if (++st == C::SP) st = 0, par ^= 1;
    };
#pragma unroll 1
    for (int u = -a.ring; u < all; ++u) {
      if (u >= 0) {  // (the first rounds only copy)
        const int rec = warp + u / UNITS * WARPS, of = rec / PER;
        if (of != now) part_done(), now = of;
        if (u % UNITS == 0 && rec - of * PER < WARPS && !tile_wait_warp(sh, a, &empty[st], par ^ 1)) return;  // (its first record of the part)
        copy_wait(a.ring - 1);
        uint32_t w[TURN][4 * WC], zs[TURN];
#pragma unroll
        for (int y = 0; y < TURN; ++y) {
#pragma unroll
          for (int e = 0; e < WC; ++e) ldsv<4>(my_codes + get * UNIT + (y * WC + e) * 512, w[y] + 4 * e);
          zs[y] = lds32(my_meta + get * UNIT + y * 128);
        }
        if (++get == a.ring) get = 0;
        // row of the part's tile; rows behind the sequence's end become zero (zero + code *
        // step = 0), whatever the page, or the place of a record that was not brought, holds
        const int at0 = (rec - of * PER) * 16 + u % UNITS * (TURN * ROWS) + row;
        const int left = p.s.len - p.blk * C::BK - of * C::PT;
        const uint32_t tile = tiles + st / (C::BK / C::PT) * C::TILE + st % (C::BK / C::PT) * (C::PT * 128);
#pragma unroll
        for (int y = 0; y < TURN; ++y) {
          uint32_t* x = w[y];
          const int at_row = at0 + y * ROWS;
          if (at_row >= left) zs[y] = 0;
          const __half2 z = __low2half2(as_h2(zs[y])), sc = __high2half2(as_h2(zs[y]));
#pragma unroll
          for (int b = 1; b < 4; b <<= 1)  // the words of chunk i to place i ^ turn
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(i & b))
#pragma unroll
                for (int e = 0; e < WC; ++e) {
                  const uint32_t lo = x[WC * i + e], hi = x[WC * (i ^ b) + e];
                  x[WC * i + e] = (turn & b) ? hi : lo;
                  x[WC * (i ^ b) + e] = (turn & b) ? lo : hi;
                }
          const uint32_t out = tile + at_row * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o[4];
            if constexpr (BITS == 8) {
              o[0] = bytes<0>(x[2 * i], sc, z);
              o[1] = bytes<1>(x[2 * i], sc, z);
              o[2] = bytes<0>(x[2 * i + 1], sc, z);
              o[3] = bytes<1>(x[2 * i + 1], sc, z);
            } else {
              o[0] = nibbles<0>(x[i], sc, z);
              o[1] = nibbles<1>(x[i], sc, z);
              o[2] = nibbles<2>(x[i], sc, z);
              o[3] = nibbles<3>(x[i], sc, z);
            }
            const int at = (4 * (piece & 1) + (i ^ turn)) ^ (at_row & 7);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(out + (at << 4)), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                         : "memory");
          }
        }
      }
      bring();  // (into the place that was read: its values have been used)
    }
    part_done();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_free[slot]));
  }
}
// Both tensors: one body where their bits are the same.
template <int D, int FMT>
__device__ __forceinline__ void tile_dequantize(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem, int value, int warp, int lane) {
  using F = typename TileCfg<D, FMT>::F;
  if constexpr (F::KB == F::VB) tile_dequantizer<D, FMT, F::KB>(a, sh, smem, value, warp, lane);
  else if (value) tile_dequantizer<D, FMT, F::VB>(a, sh, smem, 1, warp, lane);
  else tile_dequantizer<D, FMT, F::KB>(a, sh, smem, 0, warp, lane);
}

// -------------------------------------------------------------- matrix unit --

// The whole warp follows the barriers; one elected lane issues.
template <int D, int FMT, bool MASK>
__device__ __forceinline__ void tile_mma(const AttnArgs& a, TileShared<D, FMT>* sh, uint32_t smem) {
  using C = TileCfg<D, FMT>;
  constexpr uint32_t S_DESC = mma_desc(128, C::PT, C::F::kBf16, false);
  constexpr uint32_t O_DESC = mma_desc(128, D, C::F::kBf16, true);
  const uint32_t tm = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const uint64_t q0 = smem_desc(smem + C::Q_OFF, 16, 1024), k0 = smem_desc(smem + C::K_OFF, 16, 1024);
  const uint64_t v0 = smem_desc(smem + C::V_OFF, C::BK * 128, 1024);
  int ks = 0, kpar = 0, vs = 0, vpar = 0;  // part of the stages to read next, its phase
  int bc = 0;                              // score buffers handed out (one tile)
  int turns = 0;                           // phases of the weights (two tiles, a bit each)
  constexpr int HALVES = C::BK / C::PT;
  // S of a tile with the keys of part ks; O of a tile with the values of part vs (`half`:
  // which part of its block it is; the block is done with the last).
  // (Scoring the next block's first 64 keys into the columns that the weights leave
  // free, ahead of the value product, was slower: 995 us against 820 for a chunk of
  // 2048 at 32k tokens; products of 64 columns wait for shared memory.)
  auto scores = [&](int buf, int tile, int half) {
    const uint64_t q = q0 + (uint64_t)(tile * (C::TILE >> 4));
    const uint64_t k = k0 + (uint64_t)((ks / HALVES * C::TILE + half * (C::PT * 128)) >> 4);
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint64_t at = ((i >> 2) * (128 * 128) + (i & 3) * 32) >> 4;
        mma_ss(tm + buf * 128 + half * C::PT, q + at, k + at, S_DESC, i > 0);
      }
      if (half == HALVES - 1) mma_commit(smem_u32(&sh->s_full[buf]));
    }
    __syncwarp();
  };
  auto values = [&](int buf, int tile, int half, int add) {
    const uint64_t v = v0 + (uint64_t)((vs / HALVES * C::TILE + half * (C::PT * 128)) >> 4);
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < C::PT / 16; ++i)
        mma_ts(tm + 256 + tile * D, tm + buf * 128 + half * (C::PT / 2) + i * 8, v + (uint64_t)(i * 2048 >> 4), O_DESC,
               i > 0 ? 1 : add);
      if (half == HALVES - 1) mma_commit(smem_u32(&sh->o_done[tile]));
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
    if (++ks == C::SP) ks = 0, kpar ^= 1;
  };
  auto free_v = [&]() {
    if (elect_one()) mma_commit(smem_u32(&sh->v_empty[vs]));
    __syncwarp();
    if (++vs == C::SP) vs = 0, vpar ^= 1;
  };
  // (One loop from the block before a piece's first on, one copy of each product's code:
  // written out for both tiles and the first block the role was 20 KB long.)
  for (int k = 0;; ++k) {
    const int slot = k % C::PIECES;
    if (!tile_wait_warp(sh, a, &sh->piece_full[slot], (k / C::PIECES) & 1)) return;
    const int n = __shfl_sync(0xffffffffu, sh->piece[slot].nblk, 0);
    if (n == 0) return;
    if (!tile_wait_warp(sh, a, &sh->q_full, k & 1)) return;
    if (shared_rows<D, FMT, MASK>(sh->piece[slot].rows)) {
      // block j is tile j % 2's; the scores are two blocks ahead of the values
#pragma unroll 1
      for (int j = -2; j < n; ++j) {
        const int i = j & 1;
        if (j >= 0) {
          if (!tile_wait_warp(sh, a, &sh->v_full[vs], vpar)) return;
          if (!tile_wait_warp(sh, a, &sh->p_full[i], (turns >> i) & 1)) return;
          turns ^= 1 << i;
          tc_after_sync();
          values(i, i, 0, j >= 2);
          free_v();
        }
        if (j + 2 < n) {
          if (!tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
          tc_after_sync();
          scores(i, i, 0);
          free_k(j + 3 == n);
        }
      }
    } else if (C::NT == 2) {
      // the blocks that tile 0 / 1 sees
      int lo0, hi0, lo1, hi1;
      tile_range<D, FMT, MASK>(a, sh->piece[slot], 0, &lo0, &hi0);
      tile_range<D, FMT, MASK>(a, sh->piece[slot], 1, &lo1, &hi1);
      lo0 = __shfl_sync(0xffffffffu, lo0, 0);
      hi0 = __shfl_sync(0xffffffffu, hi0, 0);
      lo1 = __shfl_sync(0xffffffffu, lo1, 0);
      hi1 = __shfl_sync(0xffffffffu, hi1, 0);
#pragma unroll 1
      for (int j = -1; j < n; ++j) {
        bool have_k = false;
        if (j >= 0 && !tile_wait_warp(sh, a, &sh->v_full[vs], vpar)) return;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int lo = i ? lo1 : lo0, hi = i ? hi1 : hi0;
          if (j >= lo && j < hi) {  // (lo is not negative)
            if (!tile_wait_warp(sh, a, &sh->p_full[i], (turns >> i) & 1)) return;
            turns ^= 1 << i;
            tc_after_sync();
            values(i, i, 0, j > lo);
          }
          if (i == 1 && j >= 0) free_v();
          if (j + 1 < n && j + 1 >= lo && j + 1 < hi) {
            if (!have_k && !tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
            have_k = true;
            tc_after_sync();
            scores(i, i, 0);
          }
        }
        if (j + 1 < n) {
          if (!have_k && !tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
          free_k(j + 2 == n);
        }
      }
    } else {
#pragma unroll 1
      for (int j = -1; j < n; ++j) {
        const int buf = bc & 1;  // (the scores of block j)
        if (j + 1 < n) {
#pragma unroll 1
          for (int h = 0; h < HALVES; ++h) {
            if (!tile_wait_warp(sh, a, &sh->k_full[ks], kpar)) return;
            tc_after_sync();
            scores(j < 0 ? buf : buf ^ 1, 0, h);
            free_k(h == HALVES - 1 && j + 2 == n);
          }
        }
        if (j < 0) continue;
        if (!tile_wait_warp(sh, a, &sh->p_full[buf], (bc >> 1) & 1)) return;
#pragma unroll 1
        for (int h = 0; h < HALVES; ++h) {
          if (!tile_wait_warp(sh, a, &sh->v_full[vs], vpar)) return;
          tc_after_sync();
          values(buf, 0, h, j > 0 || h > 0);
          free_v();
        }
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
  constexpr int LPR = D / 8, RPI = 32 / LPR, U = 4;  // lanes a row, rows a step, steps in flight (16: 32 KB of code)
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

template <int D, int FMT, bool MASK>
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
    const bool dual = shared_rows<D, FMT, MASK>(p.rows);
    const int row0 = dual ? 0 : tile * 128, r = row0 + row;  // the tile's first row, the thread's
    const RowMap rm(a, p);
    const uint32_t q_tile = smem + C::Q_OFF + tile * C::TILE;
    float sc = a.scale_log2;
    if (row0 < p.rows) sc = tile_query<D, FMT>(a, rm, p.rows, row0, row & ~31, q_tile, lane);
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->q_full));
    if (row0 < p.rows) {
      const int pos = rm.position(min(r, p.rows - 1));
      // the tile's first and last position: blocks between need no mask
      const int pos_lo = MASK ? p.s.p0 - 1 : rm.position(tile * 128);
      const int pos_hi = MASK ? p.s.len - 1 : rm.position(min(tile * 128 + 127, p.rows - 1));
      int j0, j1;
      tile_range<D, FMT, MASK>(a, p, dual ? 0 : tile, &j0, &j1);
      if (dual) j0 += tile;
      float m = -INFINITY;
      float2 l = make_float2(0.0f, 0.0f);
      for (int j = j0; j < j1; j += dual ? 2 : 1, ++bc, ++ob) {
        const int buf = C::NT == 2 ? tile : (bc & 1);
        if (!tile_wait_warp(sh, a, &sh->s_full[buf], C::NT == 2 ? bc & 1 : (bc >> 1) & 1)) return;
        tc_after_sync();
        const uint32_t sb = tm + buf * 128;
        const int tok0 = (p.blk + j) * BK;
        const bool edge = tok0 + BK - 1 > pos_lo || (a.window > 0 && tok0 <= pos_hi - a.window);
        const int hi = pos - tok0, lo = a.window > 0 ? pos - a.window - tok0 : -1;  // visible columns: lo < c <= hi
        auto hide = [&](uint32_t* e, int q) {
          if constexpr (MASK) {
            const uint32_t v = seen_bits(a, p.s, rm.t0 + rm.token(min(r, p.rows - 1)), tok0 + q * 32);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(v >> c & 1)) e[c] = 0xff800000u;
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (q * 32 + c > hi || q * 32 + c <= lo) e[c] = 0xff800000u;
          }
        };
        uint32_t s[64], w[64];
        // Blocks with hidden tokens: minus infinity goes over their scores first, in a pass
        // of its own (the code of every block stays short).
        if (edge) {
#pragma unroll 1
          for (int q = 0; q < BK / 32; ++q) {
            tmem_ld32(sb + q * 32, s);
            hide(s, q);
            tmem_st32(sb + q * 32, s);
          }
          tmem_wait_st();
        }
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
      float sum = l.x + l.y;
      const bool whole = p.has_first && p.has_last, has = r < p.rows;
      // Shared rows: both tiles' maxima and sums are exchanged, and each tile puts half of
      // the columns together, from both accumulators (the same lanes of tensor memory).
      int c_lo = 0, c_hi = D;
      float f0 = 1.0f, f1 = 0.0f;
      if (dual) {
        sh->stats[tile][row & (C::NT == 2 ? 127 : 0)] = make_float2(m, sum);
        tc_before_sync();
        __syncwarp();
        uint64_t* met = &sh->met[(row >> 5) & 3];
        if (lane == 0) mbar_arrive(smem_u32(met));
        if (!tile_wait_warp(sh, a, met, 0)) return;
        tc_after_sync();
        const float2 s0 = sh->stats[0][row & (C::NT == 2 ? 127 : 0)], s1 = sh->stats[1][row & (C::NT == 2 ? 127 : 0)];
        m = fmaxf(s0.x, s1.x);
        f0 = s0.x == -INFINITY ? 0.0f : fast_exp2(s0.x - m);
        f1 = s1.x == -INFINITY ? 0.0f : fast_exp2(s1.x - m);
        sum = f0 * s0.y + f1 * s1.y;
        c_lo = tile * (D / 2), c_hi = c_lo + D / 2;
      }
      const float f = whole ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
      const long slot_row = ((long)blockIdx.x * 2 + (p.has_first ? 1 : 0)) * C::ROWS + r;
      // Whole rows go through the query tile's place (its last product is done),
      // so that the stores are D / 8 lanes a row (half as many where tiles share them).
#pragma unroll 1
      for (int c = c_lo; c < c_hi; c += 32) {
        uint32_t o[32];
        tmem_ld32(tm + (dual ? 256 : o_col) + c, o);
        if (j1 <= j0 && !dual) {  // no block: O was never written
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (dual) {
          uint32_t y[32];
          if (p.nblk > 1) tmem_ld32(tm + 256 + D + c, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float u = __uint_as_float(o[e]) * f0;
            o[e] = __float_as_uint(p.nblk > 1 ? fmaf(__uint_as_float(y[e]), f1, u) : u);
          }
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
        const int lpr = dual ? D / 16 : D / 8;  // lanes a row, iterations of 32 / lpr rows
        const int g = lane / lpr, ch = c_lo / 8 + lane % lpr;
        __syncwarp();
#pragma unroll 4
        for (int it = 0; it < lpr; ++it) {
          const int rw = (row & ~31) + it * (32 / lpr) + g;
          uint4 w;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(q_tile + (ch >> 3) * (128 * 128) + rw * 128 + (((ch & 7) ^ (rw & 7)) << 4))
                       : "memory");
          if (row0 + rw < p.rows)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + rm.at(row0 + rw, (long)a.q_heads * D, D) + ch * 8) = w;
        }
        __syncwarp();
      }
      if (!whole && has && (!dual || tile == 0)) *reinterpret_cast<float2*>(a.part_ml + slot_row * 2) = make_float2(m, sum);
      if (dual) {  // neither accumulator nor the exchanged values are written before both are done with them
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->met[(row >> 5) & 3]));
        if (!tile_wait_warp(sh, a, &sh->met[(row >> 5) & 3], 1)) return;
      }
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

template <int D, int FMT, bool MASK>
__global__ void __launch_bounds__(TileCfg<D, FMT>::THREADS, 1) pages_tile_kernel(const __grid_constant__ AttnArgs a) {
  using C = TileCfg<D, FMT>;
  using F = typename C::F;
  extern __shared__ char raw[];
  __shared__ TileShared<D, FMT> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SP; ++i) {
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
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh.met[i]), 2);
    for (int i = 0; i < C::PIECES; ++i) {
      mbar_init(smem_u32(&sh.piece_full[i]), 1);
      mbar_init(smem_u32(&sh.piece_free[i]), C::USERS);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  pdl_wait();
  plan_work<C::BK, C::ROWS, false, MASK>(a, &sh.work, reinterpret_cast<long*>(raw + C::SMEM + a.ring * C::COPIES));  // (its barriers also publish the initialisation above)
  pdl_trigger();
  if (threadIdx.x == 0) a.split[blockIdx.x].parts = 0;
  if ((int)blockIdx.x >= sh.work.ctas) return;
  if (warp == 8) tmem_alloc(smem_u32(&sh.tmem), 512);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();

  // Registers over codes: 512 threads start with 128 each (65536); two tiles take
  // 256 * 176 + 256 * 80 = 65536 of them, one tile 128 * 176 + 384 * 80 = 53248.
  if (warp < 4 * C::NT) {
    if constexpr (F::kQuant) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n");
    tile_softmax<D, FMT, MASK>(a, &sh, smem, warp >> 2, threadIdx.x);
  } else {
    if constexpr (F::kQuant) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    if (warp == 8) {
      tile_mma<D, FMT, MASK>(a, &sh, smem);
    } else if (warp == 10) {
      // the pieces of this CTA's units, ahead of the others; nblk 0 ends
      long u = cta_begin(&sh.work, blockIdx.x);
      const long end = cta_begin(&sh.work, blockIdx.x + 1);
      for (int k = 0;; ++k) {
        const int slot = k % C::PIECES;
        if (k >= C::PIECES && !tile_wait_warp(&sh, a, &sh.piece_free[slot], (k / C::PIECES - 1) & 1)) break;
        Piece p = {};
        if (u < end) {
          p = find_piece<MASK>(a, &sh.work, u, end);
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
    } else if constexpr (F::kQuant) {
      // one tile: warps 4 .. 7 values, 12 .. 15 keys; two tiles: 12, 13 and 9 keys, 14, 15 and 11 values
      if (C::NT == 1) {
        if (warp < 8 || warp >= 12) tile_dequantize<D, FMT>(a, &sh, smem, warp < 8, warp & 3, lane);
      } else {
        tile_dequantize<D, FMT>(a, &sh, smem, warp == 11 || warp >= 14, warp < 12 ? 2 : warp & 1, lane);
      }
    } else if (warp == 9) {
      tile_loader<D, FMT>(a, &sh, smem, lane);
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

template <int D, bool MASK>
AttnKernel tile_kernel_dim(int fmt) {
  switch (fmt) {
#define KVQ_TILE(f) \
  case f: return {(const void*)pages_tile_kernel<D, f, MASK>, (size_t)TileCfg<D, f>::SMEM, TileCfg<D, f>::THREADS, 0, 0, TileCfg<D, f>::COPIES};
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
