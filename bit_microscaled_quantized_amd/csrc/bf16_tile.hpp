// One 256 x 256 tile of a BF16 matrix product with FP32 accumulation on gfx950:
//   acc(m, n) = sum_k A(m, k) B(n, k)
// for operands that hold K along their rows (element (m, k) at p[m * ld + k]) or
// down their columns (KMAJOR, element (m, k) at p[k * ld + m]).
//
// 512 threads = 8 waves (two per SIMD, so that one wave's LDS reads and waits
// overlap the other's matrix instructions) in a 2 x 4 grid; wave tile 128 x 64 =
// 4 x 2 MFMA tiles of 32 x 32 x 16 (128 FP32 accumulators a lane).  A stage is
// 64 values of k: 32 KB per operand, fetched straight into LDS one stage ahead
// (two buffers, 128 KB), 16 bytes per lane, so that no registers hold data in
// flight.
//
// LDS layouts, both free of bank conflicts (64 banks of 4 bytes):
//   * K along rows: 256 rows of 128 bytes; the 16-byte chunk c of row r lies in
//     slot 8 r + (c ^ ((r >> 1) & 7)).  A fragment (row lr, 8 values of k) is one
//     16-byte read.
//   * KMAJOR: 64 rows (k) of 512 bytes; the 16-byte chunk g of row k lies in slot
//     32 k + (g ^ ((k & 3) << 2)).  A fragment is two transposing 8-byte reads
//     (ds_read_b64_tr_b16): in a block of 16 lanes, lane i names 4 values of m,
//     4 (i & 3) .., in row i >> 2, and receives those 4 rows' values at m = i.
//
// MFMA layout (32 x 32 x 16): lane l = 32 h + lr holds row lr of either operand,
// k = 8 h .. 8 h + 7; of the result, column n = lr and rows 8 (r >> 2) + 4 h +
// (r & 3), r = 0 .. 15.
//
// Addresses stay inside the operands: rows of a tile past the last are fetched
// from the last row (or, KMAJOR, from the last 8 columns) and never used.  Where
// K is not a multiple of 64 (it is one of 8), an operand with K along its rows
// gets zeros past K from the last stage; a KMAJOR operand is read up to its own
// last row of k, and one of the two must give zeros past K.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) void tile_gvoid;
typedef __attribute__((address_space(3))) void tile_lvoid;
typedef __attribute__((address_space(3))) s16x4_t tile_ls16x4;

constexpr int TILE = 256;               // both ways
constexpr int TILE_K = 64;              // values of k per stage
constexpr int TILE_OPERAND = 32 * 1024;  // bytes of an operand's stage
constexpr int TILE_STAGE = 2 * TILE_OPERAND;
constexpr int TILE_LDS = 2 * TILE_STAGE;
constexpr int TILE_THREADS = 512;

// An operand of a tile: its first element (m = the tile's first row, k = 0),
// leading dimension, and rows from there on (at least one; KMAJOR: rounded up to
// a multiple of 8, which the leading dimension covers), and, KMAJOR, how many
// values of k it holds (K or more).
struct TileOperand {
  const uint16_t* p;
  uint32_t ld;
  int rows;
  int krows;
};

// Fetch offsets (bytes) of a lane's four 16-byte loads of a stage.
template <bool KMAJOR>
struct TileFetch {
  uint32_t off[4];
  __device__ __forceinline__ void init(const TileOperand& o, int wave, int lane, int krows) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if constexpr (!KMAJOR) {
        const int r = 8 * (4 * wave + j) + (lane >> 3);
        off[j] = (uint32_t)min(r, o.rows - 1) * (o.ld * 2) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
      } else {
        const int k = 2 * (4 * wave + j) + (lane >> 5);
        const int g = (lane & 31) ^ ((k & 3) << 2);
        off[j] = (uint32_t)min(k, krows - 1) * (o.ld * 2) + 2 * min(8 * g, o.rows - 8);
      }
    }
  }
};

template <bool KMAJOR>
__device__ __forceinline__ void tile_issue(const TileOperand& o, const TileFetch<KMAJOR>& f, int kt, uint8_t* st,
                                           int wave) {
  const uint8_t* base = reinterpret_cast<const uint8_t*>(o.p) +
                        (KMAJOR ? (int64_t)kt * TILE_K * o.ld * 2 : (int64_t)kt * TILE_K * 2);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    uint32_t v = f.off[j];
    asm volatile("" : "+v"(v));  // a 32-bit offset register beside the scalar base
    __builtin_amdgcn_global_load_lds((tile_gvoid*)(base + v), (tile_lvoid*)(st + (4 * wave + j) * 1024), 16, 0, 0);
  }
}

// The last stage of an operand with K along its rows, K not a multiple of 64:
// chunks past K are zeros.
__device__ __forceinline__ void tile_last(const TileOperand& o, int kt, int K, uint8_t* st, int wave, int lane) {
  const uint8_t* base = reinterpret_cast<const uint8_t*>(o.p) + (int64_t)kt * TILE_K * 2;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int r = 8 * (4 * wave + j) + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    u32x4_t v = {0, 0, 0, 0};
    if (kt * TILE_K + 8 * c < K)
      v = *reinterpret_cast<const u32x4_t*>(base + (uint32_t)min(r, o.rows - 1) * (o.ld * 2) + 16 * c);
    *reinterpret_cast<u32x4_t*>(st + (4 * wave + j) * 1024 + lane * 16) = v;
  }
}

// Fragments of TILES MFMA tiles from row `first` of the operand's stage.
template <bool KMAJOR, int TILES>
struct TileFrag {
  uint32_t at[KMAJOR ? TILES : 1];
  uint32_t x;
  __device__ __forceinline__ void init(int first, int lane) {
    if constexpr (!KMAJOR) {
      at[0] = (uint32_t)(first + (lane & 31)) * 128;
      x = (uint32_t)((lane & 31) >> 1) & 7;
    } else {
      const int b = lane >> 4, i = lane & 15;
      x = 0;
#pragma unroll
      for (int t = 0; t < TILES; t++) {
        const int g = (((first >> 3) + 4 * t) ^ ((i >> 2) << 2)) + 2 * (b & 1) + ((i & 3) >> 1);
        at[t] = (uint32_t)(8 * (b >> 1) + (i >> 2)) * 512 + g * 16 + (i & 1) * 8;
      }
    }
  }
  __device__ __forceinline__ bf16x8_t read(const uint8_t* st, int t, int s, int h) const {
    if constexpr (!KMAJOR) {
      return *reinterpret_cast<const bf16x8_t*>(st + at[0] + t * 32 * 128 + (((2 * s + h) ^ x) << 4));
    } else {
      const uint8_t* p = st + at[t] + s * 16 * 512;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_ls16x4*)(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tile_ls16x4*)(p + 4 * 512));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// acc = the product over the stages kt0 .. kt1 - 1 (at least one) of K values
// of k.  All waves of the workgroup take part; the caller's LDS stages are free
// again after its next barrier.
template <bool AMAJ, bool BMAJ>
__device__ __forceinline__ void tile_product(const TileOperand& a, const TileOperand& b, int K, int kt0, int kt1,
                                             uint8_t* lds, floatx16 (&acc)[4][2]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5;
  TileFetch<AMAJ> fa;
  TileFetch<BMAJ> fb;
  fa.init(a, wave, lane, TILE_K);
  fb.init(b, wave, lane, TILE_K);
  TileFrag<AMAJ, 4> ra;
  TileFrag<BMAJ, 2> rb;
  ra.init((wave >> 2) * 128, lane);
  rb.init((wave & 3) * 64, lane);
  const bool ragged = (K & (TILE_K - 1)) != 0;
  const int last = (K + TILE_K - 1) / TILE_K - 1;
  // fetch of stage kt; the stage that ends past K by its own rule
  auto issue = [&](int kt, uint8_t* st) {
    if (ragged && kt == last) {
      if constexpr (AMAJ) {
        TileFetch<AMAJ> f;
        f.init(a, wave, lane, a.krows - kt * TILE_K);
        tile_issue<AMAJ>(a, f, kt, st, wave);
      } else {
        tile_last(a, kt, K, st, wave, lane);
      }
      if constexpr (BMAJ) {
        TileFetch<BMAJ> f;
        f.init(b, wave, lane, b.krows - kt * TILE_K);
        tile_issue<BMAJ>(b, f, kt, st + TILE_OPERAND, wave);
      } else {
        tile_last(b, kt, K, st + TILE_OPERAND, wave, lane);
      }
      return;
    }
    tile_issue<AMAJ>(a, fa, kt, st, wave);
    tile_issue<BMAJ>(b, fb, kt, st + TILE_OPERAND, wave);
  };
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

  bf16x8_t va[2][4], vb[2][2];
  auto read = [&](const uint8_t* st, int s, int q) {
#pragma unroll
    for (int i = 0; i < 4; i++) va[q][i] = ra.read(st, i, s, h);
#pragma unroll
    for (int j = 0; j < 2; j++) vb[q][j] = rb.read(st + TILE_OPERAND, j, s, h);
  };
  auto mma = [&](int q) {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 2; j++)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[q][i], vb[q][j], acc[i][j], 0, 0, 0);
  };

  issue(kt0, lds);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  read(lds, 0, 0);
  // One stage.  The two buffers are disjoint; restrict lets the compiler see
  // that the reads of cur do not wait for the fetch into nxt.
  auto stage = [&](int kt, const uint8_t* __restrict__ cur, uint8_t* __restrict__ nxt) {
    const bool more = kt + 1 < kt1;
    if (more) issue(kt + 1, nxt);
#pragma unroll
    for (int s = 0; s < 3; s++) {
      read(cur, s + 1, (s + 1) & 1);
      mma(s & 1);
    }
    // every wave's reads of cur are complete and its part of nxt has landed
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (more) read(nxt, 0, 0);
    mma(1);
  };
  for (int kt = kt0; kt < kt1; kt++) {
    uint8_t* cur = lds + ((kt - kt0) & 1) * TILE_STAGE;
    uint8_t* nxt = lds + ((kt - kt0 + 1) & 1) * TILE_STAGE;
    stage(kt, cur, nxt);
  }
}

// Tile (pm, pn) of workgroup bid in a grid of num_m x num_n tiles.  Workgroups
// are dealt round-robin over the 8 XCDs, so each XCD's share becomes a
// contiguous range of tiles, walked in groups of 8 tile rows, column by column,
// so that the tiles in flight on an XCD share operands in its L2.
__device__ __forceinline__ void tile_place(int bid, int num_m, int num_n, int& pm, int& pn) {
  const int G = num_m * num_n;
  const int xcd = bid & 7, per = G >> 3, rem = G & 7;
  const int id = (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + (bid >> 3);
  const int width = 8 * num_n;
  const int first = (id / width) * 8;
  const int rows = min(num_m - first, 8);
  pm = first + (id % width) % rows;
  pn = (id % width) / rows;
}

}  // namespace

}  // namespace nvfp4
