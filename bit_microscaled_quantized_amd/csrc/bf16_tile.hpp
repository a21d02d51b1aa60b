// One tile of a matrix product on gfx950, BF16 with FP32 accumulation or 8-bit
// integers with 32-bit accumulation (MfmaInt8), 256 x 256
// (W = 4), 128 x 128 (W = 2) or 64 x 64 (W = 1, K along the rows only):
//   acc(m, n) = sum_k A(m, k) B(n, k)
// for operands that hold K along their rows (element (m, k) at p[m * ld + k]) or
// down their columns (KMAJOR, element (m, k) at p[k * ld + m]).
//
// 256 threads = 4 waves, one per SIMD, in a 2 x 2 grid; wave tile of W x W MFMA
// tiles of 32 x 32 x 16 (W = 4: 256 FP32 accumulators a lane).  The chip's
// power limits this product, not its matrix rate (at full occupation of the
// matrix cores by random data the clock falls from 2.4 to 1.8 GHz), so what
// counts is energy per product: the square wave tile reads a third less from LDS
// than 8 waves of 128 x 64 (32768 x 8192 x 5120: 1.98 ms against 2.20, 1386
// against 1250 TFLOP/s).  A stage is 64 values of k: 32 KB per operand, fetched
// straight into LDS (two buffers, 128 KB; W = 2: half), 16 bytes per lane in whole 128-byte
// lines (stages of 32 values, twice as many in flight, run their 64-byte requests
// at more energy: 2.25 ms).  With one wave per SIMD nothing else hides a wait, so
// the reads and fetches are placed between the matrix instructions by hand.
// The small tile fits twice on a compute unit, so that one workgroup's start and
// end overlap the other's products: it is for products with few large tiles or
// few stages; the smallest, four to a unit, for those that have few of these too.
//
// LDS layouts, both free of bank conflicts (64 banks of 4 bytes):
//   * K along rows: rows of 128 bytes; the 16-byte chunk c of row r lies in
//     slot 8 r + (c ^ ((r >> 1) & 7)).  A fragment (row lr, 8 values of k) is one
//     16-byte read.
//   * KMAJOR: 64 rows (k) of 8 W chunks of 16 bytes; chunk g of row k lies in slot
//     8 W k + (g ^ ((k & 3) << 2)).  A fragment is two transposing 8-byte reads
//     (ds_read_b64_tr_b16): in a block of 16 lanes, lane i names 4 values of m,
//     4 (i & 3) .., in row i >> 2, and receives those 4 rows' values at m = i.
//
// MFMA layout (32 x 32 x 16): lane l = 32 h + lr holds row lr of either operand,
// k = 8 h .. 8 h + 7; of the result, column n = lr and rows 8 (r >> 2) + 4 h +
// (r & 3), r = 0 .. 15.
//
// 8-bit integers take K along the rows only, two to an element of what follows: ld,
// K and a stage's 64 count pairs, and a matrix instruction (32 x 32 x 32) reads the 16
// bytes of a lane as 16 of them.
//
// With SHIFT, K along the rows (at least a stage) may end inside a stage and the stages
// be of any number: the last stage is fetched as the K's last 64 values, and what of it
// the stage before held is cleared in the first operand; an odd number is made even by a
// stage that is all cleared.
//
// Addresses stay inside the operands: rows of a tile past the last are fetched
// from the last row (or, KMAJOR, from the last 8 columns) and never used, and a
// KMAJOR operand's values of k past its last from that one.  K along rows may end
// inside a stage (K a multiple of 8): zeros follow it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8_device.hpp"
#include "loss_device.hpp"

namespace nvfp4 {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) void tile_gvoid;
typedef __attribute__((address_space(3))) void tile_lvoid;
typedef __attribute__((address_space(3))) s16x4_t tile_ls16x4;

constexpr int TILE_K = 64;  // values of k per stage
constexpr int TILE_THREADS = 256;
constexpr int tile_side(int W) { return 64 * W; }
constexpr int tile_operand(int W) { return tile_side(W) * TILE_K * 2; }  // bytes of an operand's stage
constexpr int tile_lds(int W) { return 4 * tile_operand(W); }            // two buffers of both operands

// The matrix instruction of a tile: 16 bytes of either operand a lane.
struct MfmaBf16 {
  typedef floatx16 Acc;
  static __device__ __forceinline__ Acc mul(bf16x8_t a, bf16x8_t b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
struct MfmaInt8 {
  typedef intx16 Acc;
  static __device__ __forceinline__ Acc mul(bf16x8_t a, bf16x8_t b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(intx4, a), __builtin_bit_cast(intx4, b), c, 0, 0, 0);
  }
};

// An operand of a tile: its first element (m = the tile's first row, k = 0),
// leading dimension, and rows from there on (at least one; KMAJOR: rounded up to
// a multiple of 8, which the leading dimension covers), and, KMAJOR, how many
// values of k it holds (K or more).  once (a constant of the kernel): no other tile
// reads it, so it passes through the caches as what goes first (131072 x 5120 for
// one token: 205 us against 227).
struct TileOperand {
  const uint16_t* p;
  uint32_t ld;
  int rows;
  int krows;
  bool once = false;
};

// Fetch offsets (bytes) of a lane's 2 W 16-byte loads of a stage: load j of a wave
// fills bytes 1024 (2 W wave + j) .. of the operand's stage.
template <int W, bool KMAJOR>
struct TileFetch {
  uint32_t off[2 * W];
  uint32_t row0;  // KMAJOR: offset of load 0's row of k, the rows of a load further on per load
  static __device__ __forceinline__ int row(int wave, int lane, int j) {  // K along rows
    return 8 * (2 * W * wave + j) + (lane >> 3);
  }
  static __device__ __forceinline__ int krow(int wave, int lane, int j) {  // KMAJOR
    return ((2 * W * wave + j) * 64 + lane) / (8 * W);
  }
  // K along rows: the whole offset; KMAJOR: that of the columns
  __device__ __forceinline__ void init(const TileOperand& o, int wave, int lane) {
    row0 = (uint32_t)krow(wave, lane, 0) * (o.ld * 2);
#pragma unroll
    for (int j = 0; j < 2 * W; j++) {
      if constexpr (!KMAJOR) {
        const int r = row(wave, lane, j);
        off[j] = (uint32_t)min(r, o.rows - 1) * (o.ld * 2) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      } else {
        const int g = ((j * 64 + lane) % (8 * W)) ^ ((krow(wave, lane, j) & 3) << 2);
        off[j] = 2 * min(8 * g, o.rows - 8);
      }
    }
  }
  // load j of stage kt; not KMAJOR: that starts at value k of the rows
  __device__ __forceinline__ void issue(const TileOperand& o, int kt, int k, uint8_t* st, int wave, int j) const {
    if constexpr (KMAJOR) kt = min(kt, (o.krows - 1) / TILE_K);
    const uint8_t* base = reinterpret_cast<const uint8_t*>(o.p) +
                          (KMAJOR ? (int64_t)kt * TILE_K * o.ld * 2 : (int64_t)k * 2);
    uint32_t v = off[j];
    if constexpr (KMAJOR)  // its row of k, at most the operand's last (64 rows stay within 32 bits, all need not)
      v += min(row0 + (uint32_t)(j * (8 / W)) * (o.ld * 2),
               (uint32_t)min(o.krows - 1 - kt * TILE_K, TILE_K) * (o.ld * 2));
    asm volatile("" : "+v"(v));  // a 32-bit offset register beside the scalar base
    tile_gvoid* from = (tile_gvoid*)(base + v);
    tile_lvoid* to = (tile_lvoid*)(st + (2 * W * wave + j) * 1024);
    if (o.once)
      __builtin_amdgcn_global_load_lds(from, to, 16, 0, 2);  // non-temporal
    else
      __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
  }
};

// The last stage of an operand with K along its rows, K not a multiple of 64.
template <int W>
__device__ __forceinline__ void tile_last(const TileOperand& o, int kt, int K, uint8_t* st, int wave, int lane) {
  const uint8_t* base = reinterpret_cast<const uint8_t*>(o.p) + (int64_t)kt * TILE_K * 2;
#pragma unroll
  for (int j = 0; j < 2 * W; j++) {
    const int r = TileFetch<W, false>::row(wave, lane, j);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    u32x4_t v = {0, 0, 0, 0};
    if (kt * TILE_K + 8 * c < K)
      v = *reinterpret_cast<const u32x4_t*>(base + (uint32_t)min(r, o.rows - 1) * (o.ld * 2) + 16 * c);
    *reinterpret_cast<u32x4_t*>(st + (2 * W * wave + j) * 1024 + lane * 16) = v;
  }
}

// Fragments of the wave's W MFMA tiles from row `first` of the operand's stage.
template <int W, bool KMAJOR>
struct TileFrag {
  uint32_t at[KMAJOR ? W : 1];
  uint32_t x;
  static constexpr int ROW = 128 * W;  // bytes of a row of k (KMAJOR)
  __device__ __forceinline__ void init(int first, int lane) {
    if constexpr (!KMAJOR) {
      at[0] = (uint32_t)(first + (lane & 31)) * 128;
      x = (uint32_t)((lane & 31) >> 1) & 7;
    } else {
      const int b = lane >> 4, i = lane & 15;
      x = 0;
#pragma unroll
      for (int t = 0; t < W; t++) {
        const int g = (((first >> 3) + 4 * t) ^ ((i >> 2) << 2)) + 2 * (b & 1) + ((i & 3) >> 1);
        at[t] = (uint32_t)(8 * (b >> 1) + (i >> 2)) * ROW + g * 16 + (i & 1) * 8;
      }
    }
  }
  __device__ __forceinline__ bf16x8_t read(const uint8_t* st, int t, int s, int h) const {
    if constexpr (!KMAJOR) {
      return *reinterpret_cast<const bf16x8_t*>(st + at[0] + t * 32 * 128 + (((2 * s + h) ^ x) << 4));
    } else {
      const uint8_t* p = st + at[t] + s * 16 * ROW;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_ls16x4*)(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_ls16x4*)(p + 4 * ROW));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// Clears the first n chunks of every row of the first operand's stage.
template <int W>
__device__ __forceinline__ void tile_clear(uint8_t* st, int n) {
  const int r = threadIdx.x;
  if (r < tile_side(W))
    for (int c = 0; c < n; c++)
      *reinterpret_cast<u32x4_t*>(st + r * 128 + ((c ^ ((r >> 1) & 7)) << 4)) = u32x4_t{0, 0, 0, 0};
}

// acc = the product over the stages kt0 .. kt1 - 1 of K values of k.  EVEN: their
// number is even and K a multiple of 64 (the caller's operands hold zeros up to
// there); without it both operands have K along their rows.  All waves of the
// workgroup take part; the caller's LDS stages are free again after its next
// barrier.
template <int W, bool AMAJ, bool BMAJ, bool EVEN, typename Op = MfmaBf16, bool SHIFT = false>
__device__ __forceinline__ void tile_product(const TileOperand& a, const TileOperand& b, int K, int kt0, int kt1,
                                             uint8_t* lds, typename Op::Acc (&acc)[W][W]) {
  constexpr int OPERAND = tile_operand(W), STAGE = 2 * OPERAND;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5;
  TileFetch<W, AMAJ> fa;
  TileFetch<W, BMAJ> fb;
  static_assert(EVEN || (!AMAJ && !BMAJ), "odd stages are for K along rows");
  static_assert(!SHIFT || (EVEN && !AMAJ && !BMAJ), "a shifted stage is for K along rows");
  static_assert(W > 1 || (!AMAJ && !BMAJ), "64 columns are too few for the transposing layout");
  fa.init(a, wave, lane);
  fb.init(b, wave, lane);
  TileFrag<W, AMAJ> ra;
  TileFrag<W, BMAJ> rb;
  ra.init((wave >> 1) * 32 * W, lane);
  rb.init((wave & 1) * 32 * W, lane);
#pragma unroll
  for (int i = 0; i < W; i++)
#pragma unroll
    for (int j = 0; j < W; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0;
  bf16x8_t va[2][W], vb[2][W];

  // The stage that ends past K, and one more where the rest is odd, go first,
  // each fetched and multiplied by itself.
  int first = kt0, end = kt1;
  // where stage kt starts, and how many of its chunks are to be cleared
  auto start = [&](int kt) { return SHIFT ? min(kt * TILE_K, K - TILE_K) : kt * TILE_K; };
  auto excess = [&](int kt) { return kt >= kt1 ? 8 : max(0, (kt * TILE_K - (K - TILE_K)) / 8); };
  if constexpr (SHIFT) end += (end - first) & 1;
  if constexpr (!EVEN) {
    auto alone = [&](int kt, bool ragged) {
      if (ragged) {
        tile_last<W>(a, kt, K, lds, wave, lane);
        tile_last<W>(b, kt, K, lds + OPERAND, wave, lane);
      } else {
#pragma unroll
        for (int j = 0; j < 2 * W; j++) {
          fa.issue(a, kt, kt * TILE_K, lds, wave, j);
          fb.issue(b, kt, kt * TILE_K, lds + OPERAND, wave, j);
        }
      }
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll 1
      for (int s = 0; s < 4; s++) {
#pragma unroll
        for (int i = 0; i < W; i++) {
          va[0][i] = ra.read(lds, i, s, h);
          vb[0][i] = rb.read(lds + OPERAND, i, s, h);
        }
#pragma unroll
        for (int i = 0; i < W; i++)
#pragma unroll
          for (int j = 0; j < W; j++)
            acc[i][j] = Op::mul(va[0][i], vb[0][j], acc[i][j]);
      }
      __syncthreads();
    };
    const bool ragged = (K & (TILE_K - 1)) != 0 && kt1 * TILE_K > K;
    if (ragged) end--;
    const bool odd = ((end - first) & 1) != 0;
    if (ragged || odd) {
#pragma unroll 1
      for (int pass = 0; pass < 2; pass++) {
        if (pass == 0 ? ragged : odd) alone(pass == 0 ? end : first, pass == 0);
      }
      if (odd) first++;
    }
    if (first == end) return;
  }

  // A stage is four steps of 16 values of k, W x W matrix instructions each.  Each
  // step first reads the next step's fragments, two reads after each of its first
  // W matrix instructions (of the next stage, after the barrier that ends a stage,
  // in the last step).  A stage's loads are issued between the matrix instructions
  // of two steps: half of them as soon as their buffer is free, after that barrier,
  // half in the step after.  (All at once they keep the wave from the matrix core
  // until the address unit has taken them; later, they have not landed when the
  // stage ends.)  The last two stages' loads are clamped to the last stage, so that
  // every stage is the same code; what they fetch is not read.  The schedule
  // barriers hold the order as written.
#define TILE_FENCE __builtin_amdgcn_sched_barrier(0)
#define TILE_READ(st, s, q, x)                                 \
  do {                                                         \
    if ((x) == 0)                                              \
      va[q][0] = ra.read(st, 0, s, h);                         \
    else if ((x) <= W)                                         \
      vb[q][((x) - 1) % W] = rb.read((st) + OPERAND, ((x) - 1) % W, s, h); \
    else                                                       \
      va[q][(x) - W] = ra.read(st, (x) - W, s, h);             \
  } while (0)
#define TILE_LOAD(kt, st, x)                             \
  do {                                                   \
    if ((x) & 1)                                         \
      fb.issue(b, kt, start(kt), (st) + OPERAND, wave, (x) >> 1); \
    else                                                 \
      fa.issue(a, kt, start(kt), st, wave, (x) >> 1);    \
  } while (0)
  // fragments q in use; the next step's from step rs of rst; loads x0 .. x0 + 2 W - 1 of stage kt into dst
#define TILE_STEP(q, rst, rs, fetch, kt, dst, x0)                                                      \
  do {                                                                                                 \
    _Pragma("unroll") for (int m = 0; m < W * W; m++) {                                                \
      acc[m / W][m % W] = Op::mul(va[q][m / W], vb[q][m % W], acc[m / W][m % W]);                       \
      TILE_FENCE;                                                                                      \
      if (m < W) {                                                                                     \
        TILE_READ(rst, rs, 1 - (q), 2 * m);                                                            \
        TILE_READ(rst, rs, 1 - (q), 2 * m + 1);                                                        \
        if (W == 1 && fetch) {                                                                         \
          TILE_LOAD(kt, dst, x0);                                                                      \
          TILE_LOAD(kt, dst, (x0) + 1);                                                                \
        }                                                                                              \
      } else if (W == 4 && m < 12) {                                                                   \
        if (fetch) TILE_LOAD(kt, dst, (x0) + m - 4);                                                   \
      } else if (W == 2) {                                                                             \
        if (fetch) {                                                                                   \
          TILE_LOAD(kt, dst, (x0) + 2 * m - 4);                                                        \
          TILE_LOAD(kt, dst, (x0) + 2 * m - 3);                                                        \
        }                                                                                              \
      }                                                                                                \
      TILE_FENCE;                                                                                      \
    }                                                                                                  \
  } while (0)
  // the wait: this wave's reads of cur are complete and its part of nxt has landed
#define TILE_STAGE_OF(kt, cur, nxt)                               \
  do {                                                            \
    const int k1 = min((kt) + 1, end - 1), k2 = min((kt) + 2, end - 1); \
    TILE_STEP(0, cur, 1, true, k1, nxt, 2 * W);                       \
    TILE_STEP(1, cur, 2, false, 0, nxt, 0);                       \
    TILE_STEP(0, cur, 3, false, 0, nxt, 0);                       \
    asm volatile("" ::: "memory");                                \
    __builtin_amdgcn_s_waitcnt(0x70); /* vmcnt(0) lgkmcnt(0) */   \
    TILE_FENCE;                                                   \
    __builtin_amdgcn_s_barrier();                                 \
    TILE_FENCE;                                                   \
    asm volatile("" ::: "memory");                                \
    if constexpr (SHIFT) {                                        \
      if (excess(k1) > 0) {                                       \
        tile_clear<W>(nxt, excess(k1));                           \
        __syncthreads();                                          \
      }                                                           \
    }                                                             \
    TILE_STEP(1, nxt, 0, true, k2, cur, 0);                       \
  } while (0)
#pragma unroll
  for (int x = 0; x < 4 * W; x++) TILE_LOAD(first, lds, x);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if constexpr (SHIFT) {
    if (excess(first) > 0) {
      tile_clear<W>(lds, excess(first));
      __syncthreads();
    }
  }
#pragma unroll
  for (int x = 0; x < 2 * W; x++) TILE_READ(lds, 0, 0, x);
#pragma unroll
  for (int x = 0; x < 2 * W; x++) TILE_LOAD(first + 1, lds + STAGE, x);
  // restrict (on arguments that the compiler cannot replace by their values)
  // lets it see that reads of one buffer do not wait for the fetch into the other
  auto pair = [&](int kt, uint8_t* __restrict__ b0, uint8_t* __restrict__ b1) {
    TILE_STAGE_OF(kt, b0, b1);
    TILE_STAGE_OF(kt + 1, b1, b0);
  };
  uint32_t o0 = 0, o1 = STAGE;
  asm volatile("" : "+s"(o0), "+s"(o1));
  for (int kt = first; kt < end; kt += 2) pair(kt, lds + o0, lds + o1);
  // the clamped loads have landed before the caller uses the LDS
  __builtin_amdgcn_s_waitcnt(0);
#undef TILE_STAGE_OF
#undef TILE_STEP
#undef TILE_LOAD
#undef TILE_READ
#undef TILE_FENCE
}

// The same for a few stages, kt of them from 0 on, through one LDS buffer (half
// of tile_lds): nothing overlaps inside a workgroup, so it is for tiles of which
// several share a compute unit.
template <int W, bool AMAJ, bool BMAJ>
__device__ __forceinline__ void tile_product_short(const TileOperand& a, const TileOperand& b, int kt, uint8_t* lds,
                                                   floatx16 (&acc)[W][W]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5;
  TileFetch<W, AMAJ> fa;
  TileFetch<W, BMAJ> fb;
  fa.init(a, wave, lane);
  fb.init(b, wave, lane);
  TileFrag<W, AMAJ> ra;
  TileFrag<W, BMAJ> rb;
  ra.init((wave >> 1) * 32 * W, lane);
  rb.init((wave & 1) * 32 * W, lane);
#pragma unroll
  for (int i = 0; i < W; i++)
#pragma unroll
    for (int j = 0; j < W; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  for (int k = 0; k < kt; k++) {
    if (k > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < 2 * W; j++) {
      fa.issue(a, k, k * TILE_K, lds, wave, j);
      fb.issue(b, k, k * TILE_K, lds + tile_operand(W), wave, j);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; s++) {
      bf16x8_t va[W], vb[W];
#pragma unroll
      for (int i = 0; i < W; i++) {
        va[i] = ra.read(lds, i, s, h);
        vb[i] = rb.read(lds + tile_operand(W), i, s, h);
      }
#pragma unroll
      for (int i = 0; i < W; i++)
#pragma unroll
        for (int j = 0; j < W; j++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[i], vb[j], acc[i][j], 0, 0, 0);
    }
  }
}

// Tile (pm, pn) of workgroup bid in a grid of num_m x num_n tiles.  Workgroups
// are dealt round-robin over the 8 XCDs, so each XCD's share becomes a
// contiguous range of tiles, walked in groups of `group` tile rows, column by column,
// so that the tiles in flight on an XCD share operands in its L2.
__device__ __forceinline__ void tile_place(int bid, int num_m, int num_n, int& pm, int& pn, int group = 8) {
  const int G = num_m * num_n;
  const int xcd = bid & 7, per = G >> 3, rem = G & 7;
  const int id = (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + (bid >> 3);
  const int width = group * num_n;
  const int first = (id / width) * group;
  const int rows = min(num_m - first, group);
  pm = first + (id % width) % rows;
  pn = (id % width) / rows;
}

}  // namespace

}  // namespace nvfp4
