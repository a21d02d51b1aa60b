// A tile of the product of 8-bit integers whose stages go round three LDS buffers, so that
// two are in flight while one is multiplied: for products of so few tiles that a compute
// unit's others do not hide a fetch (bf16_tile.hpp fetches one stage ahead, in two buffers).
// Layouts of the stages and fragments, and what ends inside a stage: as there (K along
// the rows, at least a stage; its element is a pair of integers).
#pragma once

#include "bf16_tile.hpp"

namespace nvfp4 {

namespace {

constexpr int RING = 3;
constexpr int ring_lds(int W) { return RING * 2 * tile_operand(W); }

// acc = the product over the stages kt0 .. end - 1 of K pairs.  All waves of the workgroup
// take part; the LDS is free again on return.
template <int W>
__device__ __forceinline__ void ring_product(const TileOperand& a, const TileOperand& b, int K, int kt0, int end,
                                             uint8_t* lds, intx16 (&acc)[W][W]) {
  constexpr int OPERAND = tile_operand(W), STAGE = 2 * OPERAND;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  TileFetch<W, false> fa, fb;
  TileFrag<W, false> ra, rb;
  fa.init(a, wave, lane);
  fb.init(b, wave, lane);
  ra.init((wave >> 1) * 32 * W, lane);
  rb.init((wave & 1) * 32 * W, lane);
#pragma unroll
  for (int i = 0; i < W; i++)
#pragma unroll
    for (int j = 0; j < W; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0;
  // Loads of stage kt, 4 W a wave; behind the last as many, all lanes' of one place, so that
  // the wait below counts the same loads in every stage.
  auto fetch = [&](int kt, uint8_t* st) {
    const int k = min(kt * TILE_K, K - TILE_K);
#pragma unroll
    for (int j = 0; j < 2 * W; j++) {
      auto one = [&](const TileOperand& o, uint32_t off, uint8_t* to) {
        uint32_t v = kt < end ? off : 0u;
        asm volatile("" : "+v"(v));  // a 32-bit offset register beside the scalar base
        __builtin_amdgcn_global_load_lds((tile_gvoid*)(reinterpret_cast<const uint8_t*>(o.p + k) + v), (tile_lvoid*)to, 16,
                                         0, 0);
      };
      one(a, fa.off[j], st + (2 * W * wave + j) * 1024);
      one(b, fb.off[j], st + OPERAND + (2 * W * wave + j) * 1024);
    }
  };
  // Stage kt in cur, with the fetch of stage kt + 2 into dst, whose stage every wave has read
  // before the barrier.
  auto stage = [&](int kt, uint8_t* cur, uint8_t* dst) {
    constexpr int AHEAD = 4 * W * (RING - 2);  // loads of the stage behind this one
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((AHEAD & 15) | (AHEAD >> 4) << 14 | 0xF70);  // vmcnt(AHEAD): this wave's of cur have landed
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    const int excess = (kt * TILE_K - (K - TILE_K)) / 8;  // chunks that the stage before held
    if (excess > 0) {
      tile_clear<W>(cur, excess);
      __syncthreads();
    }
    fetch(kt + RING - 1, dst);
    __builtin_amdgcn_sched_barrier(0);
    bf16x8_t va[4][W], vb[4][W];
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
      for (int i = 0; i < W; i++) {
        va[s][i] = ra.read(cur, i, s, h);
        vb[s][i] = rb.read(cur + OPERAND, i, s, h);
      }
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
      for (int i = 0; i < W; i++)
#pragma unroll
        for (int j = 0; j < W; j++) acc[i][j] = MfmaInt8::mul(va[s][i], vb[s][j], acc[i][j]);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave has read cur
  };
  // restrict (on arguments that the compiler cannot replace by their values): reads of one
  // buffer do not wait for the fetches into the others
  auto round = [&](int kt, int n, uint8_t* __restrict__ b0, uint8_t* __restrict__ b1, uint8_t* __restrict__ b2) {
    stage(kt, b0, b2);
    if (n > 1) stage(kt + 1, b1, b0);
    if (n > 2) stage(kt + 2, b2, b1);
  };
  uint32_t o0 = 0, o1 = STAGE, o2 = 2 * STAGE;
  asm volatile("" : "+s"(o0), "+s"(o1), "+s"(o2));
#pragma unroll
  for (int n = 0; n < RING - 1; n++) fetch(kt0 + n, lds + n * STAGE);
  int kt = kt0;
  for (; kt + RING <= end; kt += RING) round(kt, RING, lds + o0, lds + o1, lds + o2);
  if (kt < end) round(kt, end - kt, lds + o0, lds + o1, lds + o2);
  __builtin_amdgcn_s_waitcnt(0);  // the fetches behind the last stage have landed
  __syncthreads();
}

}  // namespace

}  // namespace nvfp4
