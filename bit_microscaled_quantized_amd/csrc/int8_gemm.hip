// The product of 8-bit integers with a scale per token and per output channel
// (nvfp4_int8_gemm), for gfx950:
//   c[m][n] = (sum_k a[m][k] b[n][k]) * b_scales[n] * a_scales[m]
//
// The sum is exact in 32 bits whatever its order, so the split of K and the order
// of the tiles do not show in the result.  Tiles are those of bf16_tile.hpp on the
// 8-bit matrix instruction; the weight b is a tile's first operand, whose rows a lane
// holds four in a row of (the output's columns), so that it stores pieces of four.
// Tiles that would leave most compute units idle in a round of their own (all of them, or
// those behind the last full round) are split over K: the parts leave their integers in
// the workspace, in the order of the lanes, and a second launch adds and scales them.
//
// Large products are bound by the chip's power (8192 x 20480 x 5120: 742 us, 2315 TOP/s; 1.5
// times as fast on operands of zeros), products of some hundred tokens by the wait for each
// tile's stages and by their launches (300 x 4096 x 4096 13.5 us, 15.5 with the weight out of the caches).
#include "blocks_launch.hpp"
#include "int8_device.hpp"
#include "int8_ring.hpp"
#include "per_device.hpp"

namespace nvfp4 {

namespace {

// Place of tile t: the whole ones, and the rest, each in tile_place's order among themselves.
__device__ __forceinline__ void place(int t, int whole, int tiles, int num_n, int num_m, int& pn, int& pm) {
  const int from = t < whole ? 0 : whole, count = t < whole ? whole : tiles - whole, bid = t - from;
  const int xcd = bid & 7, per = count >> 3, rem = count & 7;
  const int id = from + (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + (bid >> 3);
  const int width = 8 * num_m, first = id / width * 8, rows = min(num_n - first, 8);
  pn = first + id % width % rows;
  pm = id % width / rows;
}

// How a tile takes its stages: an even number of whole ones, any (SHIFT), any in three
// buffers (int8_ring.hpp), or less than one.
enum Stages { kEven, kAny, kRing, kOne };

constexpr int stages_lds(int W, int stages) { return stages == kRing ? ring_lds(W) : tile_lds(W); }
// workgroups that share a compute unit, by its LDS (and, W = 4, its registers)
constexpr int per_cu(int W, int stages) {
  return W == 4 ? 1 : W == 2 ? (stages == kRing ? 1 : 2) : stages == kRing ? 3 : 4;
}

template <int W, int STAGES, typename OutT>
__global__ __launch_bounds__(TILE_THREADS, per_cu(W, STAGES)) void k_int8_tile(GemmArgs g) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int TILE = tile_side(W), WAVE = 32 * W;
  const int num_m = (g.M + TILE - 1) / TILE, num_n = (g.N + TILE - 1) / TILE, tiles = num_m * num_n;
  int t = blockIdx.x, part = 0, parts = 1;
  if (t >= g.whole) {  // neighbours take different tiles' same part
    const int rest = tiles - g.whole, u = t - g.whole;
    parts = g.parts;
    part = u / rest;
    t = g.whole + u - part * rest;
  }
  int pm, pn;
  place(t, g.whole, tiles, num_n, num_m, pn, pm);
  const int m0 = pm * TILE, n0 = pn * TILE;
  const int KT = (g.K / 2 + TILE_K - 1) / TILE_K;
  const int kt0 = (int)((int64_t)KT * part / parts), kt1 = (int)((int64_t)KT * (part + 1) / parts);
  const TileOperand wt{reinterpret_cast<const uint16_t*>(g.b + (int64_t)n0 * g.ldb), (uint32_t)(g.ldb / 2), g.N - n0, 0};
  const TileOperand tok{reinterpret_cast<const uint16_t*>(g.a + (int64_t)m0 * g.lda), (uint32_t)(g.lda / 2), g.M - m0, 0};
  intx16 acc[W][W];
  if constexpr (STAGES == kRing)
    ring_product<W>(wt, tok, g.K / 2, kt0, kt1, lds, acc);
  else
    tile_product<W, false, false, STAGES != kOne, MfmaInt8, STAGES == kAny>(wt, tok, g.K / 2, kt0, kt1, lds, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, lr = lane & 31;
  if (parts > 1) {
    intx4* out = reinterpret_cast<intx4*>(g.partial) + (int64_t)(blockIdx.x - g.whole) * (W * W * 4 * TILE_THREADS) +
                 threadIdx.x;
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int j = 0; j < W; j++)
#pragma unroll
        for (int q = 0; q < 4; q++)
          out[((i * W + j) * 4 + q) * TILE_THREADS] =
              intx4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }
  // The output leaves in whole rows of the wave's tile, through its share of the stages:
  // RB bytes of a token at a time, the 16-byte chunk c of token m in slot c ^ (m / (256 /
  // RB)), which is free of bank conflicts both ways.  (Stored as the lanes hold it, 8 bytes of
  // 32 tokens at a time, 8192 x 20480 x 5120 took 784 us, so 744.)
  constexpr int SIZE = sizeof(OutT), RB = WAVE * SIZE < 256 ? WAVE * SIZE : 256, CH = RB / 16;
  constexpr int PASSES = WAVE * SIZE / RB, IW = W / PASSES;
  __syncthreads();  // the stages are free
  uint8_t* own = lds + wave * (WAVE * RB);
  const int nb = n0 + (wave >> 1) * WAVE, mb = m0 + (wave & 1) * WAVE;
  float as[W];
#pragma unroll
  for (int j = 0; j < W; j++) as[j] = mb + lr + 32 * j < g.M ? g.a_scales[mb + lr + 32 * j] : 0.0f;
#pragma unroll
  for (int p = 0; p < PASSES; p++) {
#pragma unroll
    for (int i = 0; i < IW; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        float bs[4];
        four_scales(g, nb + 32 * (p * IW + i) + 8 * q + 4 * h, bs);
#pragma unroll
        for (int j = 0; j < W; j++) {
          const int m = 32 * j + lr, at = (32 * i + 8 * q + 4 * h) * SIZE;
          uint8_t* to = own + m * RB + (((at >> 4) ^ ((m / (256 / RB)) & (CH - 1))) << 4) + (at & 15);
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; e++) f[e] = ((float)acc[p * IW + i][j][4 * q + e] * bs[e]) * as[j];
          if constexpr (SIZE == 4)
            *reinterpret_cast<u32x4_t*>(to) = VecOf<float>::pack(f);
          else
            *reinterpret_cast<u32x2_t*>(to) = u32x2_t{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3])};
        }
      }
#pragma unroll 8
    for (int r = 0; r < WAVE; r += 64 / CH) {
      const int m = r + lane / CH, c = lane % CH;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(own + m * RB + ((c ^ ((m / (256 / RB)) & (CH - 1))) << 4));
      const int n = nb + (p * RB + c * 16) / SIZE;
      if (mb + m < g.M && n < g.N)
        store_vec<OutT>(static_cast<OutT*>(g.c) + (int64_t)(mb + m) * g.ldc + n, v, g.N - n);
    }
  }
}

// The parts' sums of one of a tile's W * W * 4 planes of pieces.
template <int W, typename OutT>
__global__ __launch_bounds__(TILE_THREADS) void k_int8_join(GemmArgs g) {
  constexpr int TILE = tile_side(W), WAVE = 32 * W, PLANES = W * W * 4;
  const int num_m = (g.M + TILE - 1) / TILE, num_n = (g.N + TILE - 1) / TILE, tiles = num_m * num_n;
  const int u = blockIdx.x / PLANES, plane = blockIdx.x % PLANES;
  int pm, pn;
  place(g.whole + u, g.whole, tiles, num_n, num_m, pn, pm);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, lr = lane & 31;
  const int i = plane / (4 * W), j = plane / 4 % W, q = plane % 4;
  const int n = pn * TILE + (wave >> 1) * WAVE + 4 * h + 32 * i + 8 * q;
  const int m = pm * TILE + (wave & 1) * WAVE + lr + 32 * j;
  if (m >= g.M || n >= g.N) return;
  const intx4* in = reinterpret_cast<const intx4*>(g.partial) + ((int64_t)u * PLANES + plane) * TILE_THREADS + threadIdx.x;
  intx4 v{0, 0, 0, 0};
#pragma unroll 4
  for (int p = 0; p < g.parts; p++) v += in[(int64_t)p * (tiles - g.whole) * PLANES * TILE_THREADS];
  float bs[4];
  four_scales(g, n, bs);
  store_four<OutT>(g, m, n, v, bs, g.a_scales[m]);
}

// The weight streams past the tokens: up to 16, and up to 64 where it is so large that its
// bytes are the time (48 x 5120 x 20480 26.4 us, 28.8 in tiles at their best parts; 64 x 4096 x
// 4096 13.2, 10.3 in tiles; 48 x 8192 x 4096, at the border, 14.1 and 13.2; 24 x 4096 x 4096 9.7 and 9.2).
bool few_tokens(int64_t M, int64_t N, int64_t K) { return M <= 16 || (M <= 64 && N * K >= (int64_t(1) << 25)); }

int64_t tiles_of(int64_t n, int W) { return (n + tile_side(W) - 1) / tile_side(W); }

constexpr int64_t slots_of(int W, bool ring) { return 256 * per_cu(W, ring ? kRing : kAny); }  // workgroups on 256 CUs

// Time of a round of `tiles` (at most slots_of) of so many stages, in microseconds, fitted
// to sweeps over the four kinds of tile and their parts (60 shapes of 64 to 16384 tokens: what it
// picks takes 0.5 % longer than the best of all in the mean, 6 % at most).  A stage takes
// longer the more of them run: of a CU's own (small tiles), of the caches and of the
// chip's power.  At their best parts W = 4, W = 2, W = 2 in three buffers and W = 1 take, in
// microseconds (M x N x K; 8192 x 20480 x 5120 747, 842 and more):
//   4096 x 5120 x 20480  380 422 500 677      1024 x 20480 x 5120  133 135 152 190
//    100 x 5120 x 20480   45  37  33  41       300 x  4096 x  4096   27  21  20  13
//   6061 x 11072 x   512   98  89 115 105
double round_us(int64_t tiles, double stages, int W, bool ring) {
  const double full = (double)tiles / (double)slots_of(W, ring);
  if (W == 4) return stages * (1.22 + 0.41 * full) + 13.5;
  if (W == 2) return ring ? stages * (0.35 + 0.28 * full) + 4.6 : stages * (0.6 + 0.46 * full) + 4.7;
  return stages * (0.22 + 0.54 * full) + 3.3;
}

struct Plan {
  int W, parts;
  bool ring;
  int64_t tiles, whole, bytes;
};
double plan_us(const Plan& p, int64_t stages) {
  const int64_t rest = p.tiles - p.whole, slots = slots_of(p.W, p.ring);
  double us = (double)(p.whole / slots) * round_us(slots, (double)stages, p.W, p.ring);
  if (p.whole % slots > 0) us += round_us(p.whole % slots, (double)stages, p.W, p.ring);
  if (rest > 0)  // and a launch that reads the parts' sums, one after the other
    us += round_us(rest * p.parts, (double)((stages + p.parts - 1) / p.parts), p.W, p.ring) + 2.8 + 0.1 * p.parts +
          (double)p.bytes * 2.0 / 6.0e6;
  return us;
}
// split false: whole tiles only
Plan plan_of(int64_t M, int64_t N, int64_t K, bool split) {
  const int64_t stages = (K / 2 + TILE_K - 1) / TILE_K;
  Plan best{0, 1, false, 0, 0, 0};
  double best_us = 0;
  for (const auto& [W, ring] : {std::pair{4, false}, {2, false}, {2, true}, {1, true}}) {
    if (K < 2 * TILE_K && W > 1) continue;
    const int64_t tiles = tiles_of(M, W) * tiles_of(N, W), slots = slots_of(W, ring);
    auto weigh = [&](const Plan& p) {
      const double us = plan_us(p, stages);
      if (best.W == 0 || us < best_us * 0.99) best = p, best_us = us;
    };
    weigh(Plan{W, 1, ring, tiles, tiles, 0});
    const int64_t whole = tiles / slots * slots, rest = tiles - whole;
    if (!split || rest == 0) continue;
    const int64_t most = std::min(slots / rest, stages / 4);
    for (int64_t parts = 2; parts <= most; parts++)
      weigh(Plan{W, (int)parts, ring, tiles, whole, parts * rest * tile_side(W) * tile_side(W) * 4});
  }
  return best;
}

template <int W, int STAGES, typename OutT>
hipError_t tile_go(const GemmArgs& g, unsigned grid, hipStream_t s) {
  constexpr int LDS = stages_lds(W, STAGES);
  if (LDS > 64 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = once_per_device(done, [] {
      return hipFuncSetAttribute(reinterpret_cast<const void*>(&k_int8_tile<W, STAGES, OutT>),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    });
    if (e != hipSuccess) return e;
  }
  k_int8_tile<W, STAGES, OutT><<<grid, TILE_THREADS, LDS, s>>>(g);
  return hipGetLastError();
}

template <int W, typename OutT>
hipError_t gemm_w(const GemmArgs& g, const Plan& p, hipStream_t s) {
  const int64_t rest = p.tiles - p.whole;
  const unsigned grid = (unsigned)(p.whole + rest * p.parts);
  hipError_t e;
  if constexpr (W == 1)
    e = g.K >= 2 * TILE_K ? tile_go<1, kRing, OutT>(g, grid, s) : tile_go<1, kOne, OutT>(g, grid, s);
  else if (W == 2 && p.ring)
    e = tile_go<2, kRing, OutT>(g, grid, s);
  else if (g.K % (4 * TILE_K) == 0 && rest == 0)
    e = tile_go<W, kEven, OutT>(g, grid, s);
  else
    e = tile_go<W, kAny, OutT>(g, grid, s);
  if (e != hipSuccess || rest == 0) return e;
  k_int8_join<W, OutT><<<(unsigned)(rest * W * W * 4), TILE_THREADS, 0, s>>>(g);
  return hipGetLastError();
}

template <typename OutT>
hipError_t gemm_t(const GemmArgs& g, const Plan& p, hipStream_t s) {
  if (p.W == 4) return gemm_w<4, OutT>(g, p, s);
  if (p.W == 2) return gemm_w<2, OutT>(g, p, s);
  return gemm_w<1, OutT>(g, p, s);
}

}  // namespace

int64_t int8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  return M == 0 ? 0 : few_tokens(M, N, K) ? few_plan(M, N, K).bytes : plan_of(M, N, K, true).bytes;
}

hipError_t launch_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* a_scales,
                            const int8_t* b, int64_t ldb, const float* b_scales, void* c, int c_dt, int64_t ldc,
                            void* workspace, int64_t workspace_bytes, hipStream_t s) {
  if (few_tokens(M, N, K)) {
    const FewPlan f = few_plan(M, N, K);
    const bool split = f.parts > 1 && workspace != nullptr && workspace_bytes >= f.bytes;
    const GemmArgs g{a,   b,   a_scales, b_scales, c, split ? static_cast<int*>(workspace) : nullptr,
                     lda, ldb, ldc, (int)M, (int)N, (int)K, 0, split ? f.parts : 1};
    return int8_few(g, c_dt, s);
  }
  Plan p = plan_of(M, N, K, true);
  if (workspace == nullptr || workspace_bytes < p.bytes) p = plan_of(M, N, K, false);
  const GemmArgs g{a,   b,   a_scales, b_scales, c, static_cast<int*>(workspace),
                   lda, ldb, ldc, (int)M, (int)N, (int)K, (int)p.whole, p.parts};
  return c_dt == 0 ? gemm_t<uint16_t>(g, p, s) : gemm_t<float>(g, p, s);
}

}  // namespace nvfp4
