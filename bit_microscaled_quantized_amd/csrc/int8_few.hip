// The product of 8-bit integers for a few tokens (nvfp4_int8_gemm; up to 64), gfx950:
// bound by reading the weight, which streams from HBM past the tokens' codes.
//
// A wave takes 16 weight rows in stages of 256 values of k.  It loads them in whole
// 128-byte lines of 8 rows, past the caches, and turns them through LDS of its own
// into MFMA fragments.  (Fragments loaded as they lie, 64 bytes of 16 rows, stream at
// 5.5 TB/s where lines reach 6.4: 20480 x 5120 read in 19.0 against 16.5 us.)  MFMA 16 x
// 16 x 64: lane l = 16 q + i holds row i of either operand, k = 16 q .. 16 q + 15; of
// the result, column i and rows 4 q + r.  The weight is the first operand, so that a
// lane has four output columns of one token.
//
// KW waves of a workgroup take a slice of K each for the same rows; RG groups of rows
// share the tokens' codes through LDS (two buffers), where there is more than one.
// LDS layout of either: rows of 256 bytes, the 16-byte chunk c of row r in slot c ^ (r &
// 15), free of bank conflicts.  Where the workgroups are too few, K is split over them
// as well: parts leave their integers in the workspace and a second launch adds and
// scales them.
#include <algorithm>

#include "blocks_launch.hpp"
#include "int8_device.hpp"

namespace nvfp4 {

namespace {

constexpr int STAGE = 256;  // values of k

// 16 bytes at a 32-bit offset from a base that is the same for the wave.  ONCE: past the
// caches.
template <bool ONCE>
__device__ __forceinline__ intx4 load16(const int8_t* base, uint32_t off) {
  const intx4* p = reinterpret_cast<const intx4*>(base + off);
  return ONCE ? __builtin_nontemporal_load(p) : *p;
}
// Offset of chunk c of row r
__device__ __forceinline__ int slot(int r, int c) { return r * STAGE + ((c ^ (r & 15)) << 4); }

// MT: tiles of 16 tokens.
template <int MT, int RG, int KW, typename OutT>
__global__ __launch_bounds__(64 * RG * KW) void k_int8_few(GemmArgs g) {
  constexpr bool SHARED = RG > 1;
  static_assert(RG == 1 || (RG == 4 && KW == 1), "a row of 16 chunks of tokens to 16 threads");
  constexpr int TOK = SHARED ? 16 * MT * STAGE : 0;  // a buffer of tokens
  extern __shared__ __align__(16) int8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rg = wave % RG, kw = wave / RG;
  int8_t* own = lds + 2 * TOK + wave * (16 * STAGE);
  const int blocks = (g.N + 16 * RG - 1) / (16 * RG);
  const int part = blockIdx.x / blocks, block = blockIdx.x - part * blocks;
  const int n0 = (block * RG + rg) * 16;
  const int stages = (g.K + STAGE - 1) / STAGE;
  const int slices = g.parts * KW, slice = part * KW + kw;
  const int first = (int)((int64_t)stages * slice / slices), end = (int)((int64_t)stages * (slice + 1) / slices);
  // load j of a stage: rows 8 (j & 1) + lane / 8, chunks 8 (j >> 1) + lane % 8.  Rows past
  // the last are read from the last, whose results are not stored.
  const int nb = min(n0, g.N - 1);
  const int8_t* base = g.b + (int64_t)nb * g.ldb;
  uint32_t ob[2];
#pragma unroll
  for (int j = 0; j < 2; j++) ob[j] = (uint32_t)min(8 * j + (lane >> 3), g.N - 1 - nb) * (uint32_t)g.ldb;
  // tokens: own fragments, or a lane's share of a stage, chunk tid % 16 of rows tid / 16 + 16 t
  constexpr int TA = MT;
  uint32_t oa[TA];
#pragma unroll
  for (int t = 0; t < TA; t++) oa[t] = (uint32_t)min(16 * t + (SHARED ? tid >> 4 : i), g.M - 1) * (uint32_t)g.lda;
  intx4 acc[MT], vb[4], va[SHARED ? TA : 4 * TA];
#pragma unroll
  for (int t = 0; t < MT; t++) acc[t] = intx4{0, 0, 0, 0};
  // Loads of stage kt.  The last one may end inside: its last chunk stands for those past K,
  // and the weight's are cleared as they are put into LDS.  Waves that share tokens load on no
  // condition, behind their slice's end all lanes from one place, so that the compiler waits for
  // a stage with the next one's loads in flight (48 tokens of 20480 x 5120 28.8 against
  // 30.1 us; a stage more in flight gained nothing).  Waves on their own hide each
  // other's waits (131072 x 5120 96 us, 99 with loads on no condition).
  auto offset = [&](uint32_t row, int kt, int col) {
    return !SHARED || kt < end ? row + (uint32_t)min(STAGE * kt + col, g.K - 16) : 0u;
  };
  auto load_b = [&](int kt) {
    if (!SHARED && kt >= end) return;
#pragma unroll
    for (int j = 0; j < 4; j++) vb[j] = load16<true>(base, offset(ob[j & 1], kt, 128 * (j >> 1) + 16 * (lane & 7)));
  };
  auto put_b = [&](int kt) {
    if (STAGE * (kt + 1) > g.K) {
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (STAGE * kt + 128 * (j >> 1) + 16 * (lane & 7) >= g.K) vb[j] = intx4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
      *reinterpret_cast<intx4*>(own + slot(8 * (j & 1) + (lane >> 3), 8 * (j >> 1) + (lane & 7))) = vb[j];
  };
  auto load_a = [&](int kt) {
    if (!SHARED && kt >= end) return;
#pragma unroll
    for (int t = 0; t < TA; t++) {
      if constexpr (SHARED) {
        va[t] = load16<false>(g.a, offset(oa[t], kt, 16 * (tid & 15)));
      } else {
#pragma unroll
        for (int s = 0; s < 4; s++) va[s * TA + t] = load16<false>(g.a, offset(oa[t], kt, 64 * s + 16 * q));
      }
    }
  };
  auto put_a = [&](int buf) {
    if constexpr (SHARED) {
#pragma unroll
      for (int t = 0; t < TA; t++)
        *reinterpret_cast<intx4*>(lds + buf * TOK + slot(16 * t + (tid >> 4), tid & 15)) = va[t];
    }
  };
  load_a(first);
  load_b(first);
  if constexpr (SHARED) {
    put_a(0);
    load_a(first + 1);
    __syncthreads();
  }
  for (int kt = first; kt < end; kt++) {
    const int buf = (kt - first) & 1;
    put_b(kt);
    load_b(kt + 1);
    if constexpr (SHARED) {
      put_a(buf ^ 1);
      load_a(kt + 2);
    }
#pragma unroll
    for (int s = 0; s < 4; s++) {
      const intx4 fb = *reinterpret_cast<const intx4*>(own + slot(i, 4 * s + q));
#pragma unroll
      for (int t = 0; t < MT; t++) {
        intx4 fa;
        if constexpr (SHARED)
          fa = *reinterpret_cast<const intx4*>(lds + buf * TOK + slot(16 * t + i, 4 * s + q));
        else
          fa = va[s * TA + t];
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb, fa, acc[t], 0, 0, 0);
      }
    }
    if constexpr (SHARED)
      __syncthreads();
    else
      load_a(kt + 1);
  }
  // slices of K meet in LDS
  if constexpr (KW > 1) {
    intx4* sums = reinterpret_cast<intx4*>(lds);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; t++) sums[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
      for (int w = 1; w < KW; w++) acc[t] += sums[((w * RG + rg) * MT + t) * 64 + lane];
  }
  if (g.partial != nullptr) {
    intx4* out = reinterpret_cast<intx4*>(g.partial) + (int64_t)blockIdx.x * (MT * RG * 64) + rg * 64 + lane;
#pragma unroll
    for (int t = 0; t < MT; t++) out[t * (RG * 64)] = acc[t];
    return;
  }
  const int n = n0 + 4 * q;
  float bs[4];
  four_scales(g, n, bs);
#pragma unroll
  for (int t = 0; t < MT; t++) {
    const int m = 16 * t + i;
    if (m < g.M && n < g.N) store_four<OutT>(g, m, n, acc[t], bs, g.a_scales[m]);
  }
}

// The parts' sums of one of a block's MT planes of pieces.
template <int MT, int RG, typename OutT>
__global__ __launch_bounds__(64 * RG) void k_int8_few_join(GemmArgs g) {
  const int blocks = (g.N + 16 * RG - 1) / (16 * RG);
  const int block = blockIdx.x / MT, t = blockIdx.x % MT;
  const int lane = threadIdx.x & 63, rg = threadIdx.x >> 6;
  const int n = (block * RG + rg) * 16 + 4 * (lane >> 4), m = 16 * t + (lane & 15);
  if (m >= g.M || n >= g.N) return;
  const intx4* in = reinterpret_cast<const intx4*>(g.partial) + ((int64_t)block * MT + t) * (RG * 64) + threadIdx.x;
  intx4 v{0, 0, 0, 0};
#pragma unroll 4
  for (int p = 0; p < g.parts; p++) v += in[(int64_t)p * blocks * (MT * RG * 64)];
  float bs[4];
  four_scales(g, n, bs);
  store_four<OutT>(g, m, n, v, bs, g.a_scales[m]);
}

template <int MT, int RG, int KW, typename OutT>
hipError_t few_t(const GemmArgs& g, hipStream_t s) {
  constexpr int LDS = RG * KW * 16 * STAGE + (RG > 1 ? 2 * 16 * MT * STAGE : 0);
  static_assert(LDS <= 64 * 1024 && KW * RG * MT * 1024 <= LDS, "LDS of a workgroup");
  const unsigned blocks = (unsigned)((g.N + 16 * RG - 1) / (16 * RG));
  k_int8_few<MT, RG, KW, OutT><<<blocks * g.parts, 64 * RG * KW, LDS, s>>>(g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.parts == 1) return e;
  k_int8_few_join<MT, RG, OutT><<<blocks * MT, 64 * RG, 0, s>>>(g);
  return hipGetLastError();
}

// Groups of rows and slices of K of a workgroup.  Few tokens are read from the caches by
// each wave for itself (a token of 20480 x 5120 18.3 us, shared 22.8; 8 tokens 19.6
// against 21.7, 16 level), which for up to 16 also saves the second launch where the
// weight is small (16 tokens of 1024 x 5120 5.9 us against 8.3, of 5120 x 5120 9.9 against
// 9.9, of 20480 x 5120 23.3 against 22.1).
struct Shape {
  int rg, kw;
};
Shape shape_of(int64_t M, int64_t N, int64_t K) {
  if (M > 16 || (M > 8 && N * K > (int64_t(1) << 25))) return Shape{4, 1};
  return Shape{1, N >= 16 * 640 ? 4 : 8};
}

template <typename OutT>
hipError_t few(const GemmArgs& g, hipStream_t s) {
  const Shape f = shape_of(g.M, g.N, g.K);
  if (f.rg == 1) return f.kw == 4 ? few_t<1, 1, 4, OutT>(g, s) : few_t<1, 1, 8, OutT>(g, s);
  switch ((g.M + 15) / 16) {
    case 1: return few_t<1, 4, 1, OutT>(g, s);
    case 2: return few_t<2, 4, 1, OutT>(g, s);
    case 3: return few_t<3, 4, 1, OutT>(g, s);
    default: return few_t<4, 4, 1, OutT>(g, s);
  }
}

}  // namespace

// K is split over workgroups until there are two on each of 256 CUs of those that share tokens
// (48 tokens of 5120 x 20480 26.9 us in six parts, 28.4 in eight; 32 tokens of 20480 x 5120, 320
// workgroups already, 26.3 in two, 27.3 in one, but 48 level), with two stages or more;
// waves on their own, 5120 in all with two stages, where they would have eight or more (a
// token of 5120 x 20480 20.7 us in four parts, 28 in one).
FewPlan few_plan(int64_t M, int64_t N, int64_t K) {
  const Shape f = shape_of(M, N, K);
  const int64_t blocks = (N + 16 * f.rg - 1) / (16 * f.rg), stages = (K + STAGE - 1) / STAGE;
  int64_t parts = 1;
  if (f.rg > 1)
    parts = std::min((blocks > 256 && M <= 32 ? 640 : 512) / blocks, stages / 2);
  else if (stages >= 8 * f.kw)
    parts = std::min(5120 / (blocks * f.kw), stages / (2 * f.kw));
  parts = std::max<int64_t>(parts, 1);
  return FewPlan{(int)parts, parts == 1 ? 0 : parts * blocks * 16 * f.rg * ((M + 15) / 16 * 16) * 4};
}

hipError_t int8_few(const GemmArgs& g, int c_dt, hipStream_t s) {
  return c_dt == 0 ? few<uint16_t>(g, s) : few<float>(g, s);
}

}  // namespace nvfp4
