// Softmax cross entropy of a linear head and its gradient
// (nvfp4_linear_cross_entropy, nvfp4_linear_cross_entropy_backward), gfx950.
//
// Forward: the logits z = x W^T are formed in tiles on the BF16 matrix
// cores (bf16_tile.hpp); each tile leaves one (maximum, sum of exp(z - maximum))
// pair per token, and the label's logit; a second kernel joins a token's pairs.
// Backward, on the tokens that have a label only, over pieces of the vocabulary:
// the logits tile is formed again, d = dloss (exp(z - lse) - [v = label]) is held
// as BF16 for the piece (in what units, and when in two parts: Tokens, loss_device.hpp), and two products follow: dW = d^T x (whole per piece)
// and dx += d W (FP32 in the workspace across pieces, rounded to BF16 once).
//
// Every product has its output's contiguous dimension as the tile's rows m, so a
// lane holds four consecutive values of an output row (or 64 logits of each of
// four tokens): the operands are fetched in whichever orientation they lie in
// memory, and nothing is transposed in HBM.
//   logits      m vocabulary (W, k along rows)    n tokens (x, k along rows)
//   d^T[v][t]   m tokens (x, k along rows)        n vocabulary (W, k along rows)
//   dW[v][h]    m hidden (x, k down columns)      n vocabulary (d^T, k along rows)
//   dx[t][h]    m hidden (W, k down columns)      n tokens (d^T, k down columns)
#include "bf16_tile.hpp"
#include "layers_launch.hpp"
#include "loss_device.hpp"
#include "per_device.hpp"

namespace nvfp4 {

namespace {

// Row m of the tile of register r of MFMA tile i, without the lane's 4 h.
__device__ __forceinline__ int tile_row(int i, int r) { return 32 * i + 8 * (r >> 2) + (r & 3); }

// stats[t][vt] = the pair of token t and vocabulary tile vt; zlab[t] = the
// logit of t's label.
template <int W, bool EVEN, bool ONCE>
__global__ __launch_bounds__(TILE_THREADS, W == 4 ? 1 : W == 2 ? 2 : 4) void k_logits_stats(const uint16_t* w, uint32_t ld_w, int V,
                                                                  const uint16_t* x, uint32_t ld_x, int T, int H,
                                                                  const int64_t* labels, float2* stats, float* zlab) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int TILE = tile_side(W), WAVE = 32 * W;
  int pm, pn;
  tile_place(blockIdx.x, (V + TILE - 1) / TILE, (T + TILE - 1) / TILE, pm, pn);
  const int m0 = pm * TILE, n0 = pn * TILE;
  floatx16 acc[W][W];
  tile_product<W, false, false, EVEN>(TileOperand{w + (int64_t)m0 * ld_w, ld_w, V - m0, H, ONCE},
                             TileOperand{x + (int64_t)n0 * ld_x, ld_x, T - n0, H}, H, 0, (H + TILE_K - 1) / TILE_K, lds,
                             acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  const int rows = V - m0 - wm * WAVE - 4 * h;  // vocabulary rows from the lane's first
  float2 st[W];
#pragma unroll
  for (int j = 0; j < W; j++) {
    st[j] = make_float2(-INFINITY, 0.0f);
    if (n0 + wn * WAVE + 32 * j >= T) continue;  // no tokens here
    const int t = n0 + wn * WAVE + 32 * j + lr;
    if (V - m0 < TILE) {
#pragma unroll
      for (int i = 0; i < W; i++)
#pragma unroll
        for (int r = 0; r < 16; r++)
          if (tile_row(i, r) >= rows) acc[i][j][r] = -INFINITY;  // adds nothing below
    }
    // the label's row from the lane's first, where it is one of the wave's
    const int64_t label = t < T ? labels[t] : -1;
    const int lab = label >= 0 && label < V ? (int)label - m0 - wm * WAVE - 4 * h : -1;
    if (__any(lab >= 0 && lab < WAVE)) {
      float z = 0.0f;
      bool mine = false;  // rows alternate in fours between the lanes of a column
#pragma unroll
      for (int i = 0; i < W; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
          z = lab == tile_row(i, r) ? acc[i][j][r] : z;
          mine = mine || lab == tile_row(i, r);
        }
      if (mine) zlab[t] = z;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) mx = fmaxf(mx, acc[i][j][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float sh = shift_of(mx);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) s += exp_fast(acc[i][j][r] - sh);
    s += __shfl_xor(s, 32, 64);
    st[j] = make_float2(mx, s);
  }
  // join the two waves of a column, in LDS (the stages are free)
  __syncthreads();
  float2* half = reinterpret_cast<float2*>(lds);
  if (wm == 1 && h == 0)
    for (int j = 0; j < W; j++) half[wn * WAVE + 32 * j + lr] = st[j];
  __syncthreads();
  if (wm == 0 && h == 0)
    for (int j = 0; j < W; j++) {
      const int t = n0 + wn * WAVE + 32 * j + lr;
      if (t < T) stats[(int64_t)t * ((V + TILE - 1) / TILE) + pm] = join(st[j], half[wn * WAVE + 32 * j + lr]);
    }
}

// lse and loss of a token from its `tiles` pairs: one workgroup per token.
__global__ __launch_bounds__(256) void k_loss(const float2* stats, int tiles, int V, const int64_t* labels,
                                              const float* zlab, float* loss, float* lse) {
  __shared__ float2 part[4];
  const int64_t t = blockIdx.x;
  float2 st = make_float2(-INFINITY, 0.0f);
  for (int q = threadIdx.x; q < tiles; q += 256) st = join(st, stats[t * tiles + q]);
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) st = join(st, make_float2(__shfl_xor(st.x, m, 64), __shfl_xor(st.y, m, 64)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = st;
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int q = 1; q < 4; q++) st = join(st, part[q]);
  const float l = st.x + logf(st.y);
  lse[t] = l;
  const int64_t lab = labels[t];
  loss[t] = lab >= 0 && lab < V ? l - zlab[t] : 0.0f;
}

// ---- backward: the tokens that have a label come first

// The unit of d: 1 where the largest |dloss| m is no normal number (an infinity's quotients are NaN).
__device__ __forceinline__ float scale_of(float m) { return m >= 0x1p-126f && m < INFINITY ? m : 1.0f; }

// One workgroup: token t's place is the number of labelled tokens before it.
__global__ __launch_bounds__(1024) void k_tokens(const int64_t* labels, const float* dloss, int64_t T, int64_t V,
                                                 Tokens tk) {
  __shared__ int sums[1024];
  __shared__ float tops[16];
  const int tid = threadIdx.x;
  const int64_t per = (T + 1023) / 1024, t0 = min(T, tid * per), t1 = min(T, t0 + per);
  int c = 0;
  float top = 0.0f;
  for (int64_t t = t0; t < t1; t++)
    if (labels[t] >= 0 && labels[t] < V) {
      c++;
      top = fmaxf(top, __builtin_fabsf(dloss[t]));
    }
  sums[tid] = c;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = tid >= o ? sums[tid - o] : 0;
    __syncthreads();
    sums[tid] += v;
    __syncthreads();
  }
  int at = sums[tid] - c;
  for (int64_t t = t0; t < t1; t++) {
    const bool valid = labels[t] >= 0 && labels[t] < V;
    tk.place[t] = valid ? at : -1;
    if (valid) tk.list[at++] = (int)t;
  }
  if (tid != 1023) return;
  *tk.n = sums[1023];
  for (int q = 0; q < 16; q++) top = fmaxf(top, tops[q]);
  *tk.scale = scale_of(top);
}

// k_tokens and k_gather for up to FEW_LABELS tokens, one launch: every workgroup
// counts the labels itself (those before its 4 tokens, and all of them); a wave copies
// a token.
constexpr int64_t FEW_LABELS = 4096;
__global__ __launch_bounds__(256) void k_tokens_gather(const int64_t* labels, const float* dloss, int T, int64_t V,
                                                       const uint16_t* x, int64_t ld_x, int64_t H, Tokens tk,
                                                       uint16_t* xc) {
  __shared__ int part[2][4];
  __shared__ float tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, first = blockIdx.x * 4;
  auto labelled = [&](int t) { return t < T && labels[t] >= 0 && labels[t] < V; };
  int before = 0, all = 0;
  float top = 0.0f;
  const uint64_t mine = __ballot(lane < 4 && labelled(first + lane));  // of the workgroup's tokens
  for (int t = tid; t < T; t += 256) {
    const int v = labelled(t) ? 1 : 0;
    all += v;
    before += t < first ? v : 0;
    if (v != 0 && blockIdx.x == 0) top = fmaxf(top, __builtin_fabsf(dloss[t]));
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    all += __shfl_xor(all, m, 64);
    before += __shfl_xor(before, m, 64);
    top = fmaxf(top, __shfl_xor(top, m, 64));
  }
  if ((tid & 63) == 0) {
    part[0][tid >> 6] = before;
    part[1][tid >> 6] = all;
    tops[tid >> 6] = top;
  }
  __syncthreads();
  const int n = part[1][0] + part[1][1] + part[1][2] + part[1][3];
  const bool two = n <= tk.half;
  const int cols = n == 0 ? 0 : two ? tk.half + n : n;
  if (blockIdx.x == 0 && tid == 0) {
    *tk.n = n;
    *tk.scale = scale_of(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
  }
  const int t = first + wave;
  const bool valid = (mine >> wave) & 1;
  const int at = part[0][0] + part[0][1] + part[0][2] + part[0][3] + __popcll(mine & ((1u << wave) - 1));
  if (lane == 0 && t < T) {
    tk.place[t] = valid ? at : -1;
    if (valid) tk.list[at] = t;
  }
  if (valid) {
#pragma unroll 4
    for (int64_t c = lane * 8; c < H; c += 64 * 8) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + t * ld_x + c);
      *reinterpret_cast<u32x4_t*>(xc + at * H + c) = v;
      if (two) *reinterpret_cast<u32x4_t*>(xc + (tk.half + at) * H + c) = v;
    }
  }
  // the grid covers T up to a multiple of 128: rows without a token are zeros where K needs them
  if (t >= n && t < (cols + 127) / 128 * 128 && !(two && t >= tk.half && t < cols))
    for (int64_t c = lane * 8; c < H; c += 64 * 8) *reinterpret_cast<u32x4_t*>(xc + t * H + c) = u32x4_t{0, 0, 0, 0};
}

// xc[i] = x[list[i]] for the n labelled tokens (nothing else of x is read
// again), twice where d has two parts, and zeros elsewhere up to a multiple of 128
// rows (K of the dw product).
__global__ __launch_bounds__(256) void k_gather(const uint16_t* x, int64_t ld_x, int64_t H, Tokens tk, uint16_t* xc) {
  const int64_t i = blockIdx.x;
  const int n = *tk.n, cols = tk.columns();
  if (i >= (cols + 127) / 128 * 128) return;
  const int64_t at = tk.two() && i >= tk.half ? i - tk.half : i;
  const uint16_t* src = x + (at < n ? (int64_t)tk.list[at] * ld_x : 0);
  for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8)
    *reinterpret_cast<u32x4_t*>(xc + i * H + c) =
        at < n ? *reinterpret_cast<const u32x4_t*>(src + c) : u32x4_t{0, 0, 0, 0};
}

// ---- a BF16 tile through LDS: rows n of 64 W values of m (8 W chunks of 16
// bytes); chunk g of row n lies in slot g ^ (n mod 8 W), so that the rows a wave
// writes at once fall into different banks.

// Four consecutive values of m (from 8 g + 4 half) of row n.
template <int W>
__device__ __forceinline__ void tile_put(uint8_t* lds, int n, int g, int half, uint32_t lo, uint32_t hi) {
  *reinterpret_cast<u32x2_t*>(lds + n * 128 * W + ((g ^ (n & (8 * W - 1))) << 4) + 8 * half) = u32x2_t{lo, hi};
}
template <int W>
__device__ __forceinline__ u32x4_t tile_get(const uint8_t* lds, int n, int g) {
  return *reinterpret_cast<const u32x4_t*>(lds + n * 128 * W + ((g ^ (n & (8 * W - 1))) << 4));
}

// What a value's BF16 leaves of it (nothing where that is infinite).
__device__ __forceinline__ float rest(float v, float held) {
  return __builtin_fabsf(held) == INFINITY ? 0.0f : v - held;
}

// d^T of a piece of the vocabulary, BF16 [rows up to a multiple of 128][ldd], one
// column per labelled token (or two, see Tokens), zeros in the other columns up to a
// multiple of 128 and in the rows past the piece's last: both are K of a later product.
template <int W, bool EVEN, bool ONCE>
__global__ __launch_bounds__(TILE_THREADS, W == 4 ? 1 : W == 2 ? 2 : 4) void k_logits_grad(const uint16_t* w, uint32_t ld_w, int rows,
                                                                 const uint16_t* xc, int H, int tiles_t, int64_t v_first,
                                                                 Tokens tk, const int64_t* labels, const float* lse,
                                                                 const float* dloss, uint16_t* d, int64_t ldd) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int TILE = tile_side(W), WAVE = 32 * W;
  const int n_tok = *tk.n;
  const int padded = (rows + 127) / 128 * 128;
  int pm, pn;  // token tile, vocabulary tile
  tile_place(blockIdx.x, tiles_t, (padded + TILE - 1) / TILE, pm, pn);
  const int m0 = pm * TILE, n0 = pn * TILE;
  const bool two = n_tok <= tk.half;  // then the first tile of tokens holds all, and writes both parts
  if (m0 >= (two ? min(n_tok, 1) : (n_tok + 127) / 128 * 128)) return;
  // Columns first .. end - 1 of d^T from the tile in LDS, which starts with token m0.
  auto store = [&](int first, int end) {
    for (int e = threadIdx.x; e < TILE * 8 * W; e += TILE_THREADS) {
      const int n = e / (8 * W), g = e % (8 * W);
      const int c = first + 8 * g, left = n_tok - m0 - 8 * g;  // tokens from this column on
      if (n0 + n >= padded || c >= end) continue;
      u32x4_t v = {0, 0, 0, 0};
      if (n0 + n < rows && left > 0) {
        v = tile_get<W>(lds, n, g);
        if (left < 8) {
#pragma unroll
          for (int k = 0; k < 4; k++) v[k] &= (2 * k < left ? 0xFFFFu : 0u) | (2 * k + 1 < left ? 0xFFFF0000u : 0u);
        }
      }
      *reinterpret_cast<u32x4_t*>(d + (int64_t)(n0 + n) * ldd + c) = v;
    }
  };
  if (W == 1 && (m0 >= n_tok || n0 >= rows)) {  // only zeros
    store(m0, two ? tk.half : (int)ldd);
    if (two) store(tk.half, (int)ldd);
    return;
  }
  floatx16 acc[W][W];
  tile_product<W, false, false, EVEN>(TileOperand{xc + (int64_t)m0 * H, (uint32_t)H, n_tok - m0, H},
                             TileOperand{w + (int64_t)n0 * ld_w, ld_w, rows - n0, H, ONCE}, H, 0, (H + TILE_K - 1) / TILE_K, lds,
                             acc);
  // what the tile's tokens hold: lse, dloss, and the label's row in this tile (or -1)
  __syncthreads();
  float* s_lse = reinterpret_cast<float*>(lds + tile_lds(W));
  float* s_g = s_lse + TILE;
  int* s_lab = reinterpret_cast<int*>(s_g + TILE);
  if (threadIdx.x < TILE) {
    const int i = m0 + threadIdx.x;
    float l = 0.0f, g = 0.0f;
    int64_t lab = -1;
    if (i < n_tok) {
      const int t = tk.list[i];
      l = lse[t];
      g = dloss[t] / *tk.scale;
      lab = labels[t] - v_first - n0;
    }
    s_lse[threadIdx.x] = l;
    s_g[threadIdx.x] = g;
    s_lab[threadIdx.x] = lab >= 0 && lab < TILE ? (int)lab : -1;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  // a label of the wave's tokens among its vocabulary rows?  (-1 stays -1)
  const int lab0 = s_lab[wm * WAVE + (lane & (WAVE - 1))], lab1 = s_lab[wm * WAVE + WAVE - 1 - (lane & (WAVE - 1))];
  const bool hit = __any((lab0 >= 0 && lab0 / WAVE == wn) || (lab1 >= 0 && lab1 / WAVE == wn));
  // PART 1: what BF16 leaves of d
  auto put = [&](auto with_labels, auto part) {
#pragma unroll
    for (int i = 0; i < W; i++) {
      if (m0 + wm * WAVE + 32 * i >= n_tok) continue;  // no tokens here
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = wm * WAVE + 32 * i + 8 * q + 4 * h;
        const float4 l = *reinterpret_cast<const float4*>(s_lse + m);
        const float4 g = *reinterpret_cast<const float4*>(s_g + m);
        int4 lab = make_int4(-1, -1, -1, -1);
        if constexpr (with_labels.value) lab = *reinterpret_cast<const int4*>(s_lab + m);
#pragma unroll
        for (int j = 0; j < W; j++) {
          const int n = wn * WAVE + 32 * j + lr;
          float p0 = exp_fast(acc[i][j][4 * q] - l.x), p1 = exp_fast(acc[i][j][4 * q + 1] - l.y);
          float p2 = exp_fast(acc[i][j][4 * q + 2] - l.z), p3 = exp_fast(acc[i][j][4 * q + 3] - l.w);
          if constexpr (with_labels.value) {
            p0 -= lab.x == n ? 1.0f : 0.0f;
            p1 -= lab.y == n ? 1.0f : 0.0f;
            p2 -= lab.z == n ? 1.0f : 0.0f;
            p3 -= lab.w == n ? 1.0f : 0.0f;
          }
          p0 *= g.x, p1 *= g.y, p2 *= g.z, p3 *= g.w;
          uint32_t d01 = bf16_pack(p0, p1), d23 = bf16_pack(p2, p3);
          if constexpr (part.value == 1) {
            d01 = bf16_pack(rest(p0, bf16lo(d01)), rest(p1, bf16hi(d01)));
            d23 = bf16_pack(rest(p2, bf16lo(d23)), rest(p3, bf16hi(d23)));
          }
          tile_put<W>(lds, n, m >> 3, h, d01, d23);
        }
        __builtin_amdgcn_sched_barrier(0);  // few token values at a time beside 256 accumulators
      }
    }
  };
  using std::integral_constant;
  if (two) {
    put(std::true_type{}, integral_constant<int, 0>{});
    __syncthreads();
    store(m0, tk.half);
    __syncthreads();
    put(std::true_type{}, integral_constant<int, 1>{});
    __syncthreads();
    store(tk.half, (int)ldd);
    return;
  }
  if (hit)
    put(std::true_type{}, integral_constant<int, 0>{});
  else
    put(std::false_type{}, integral_constant<int, 0>{});
  __syncthreads();
  store(m0, (int)ldd);
}

// dw[v][h] (+)= sum over the labelled tokens of d^T[v][i] xc[i][h]
template <int W, bool SHORT, bool STREAM, typename OutT>
__global__ __launch_bounds__(TILE_THREADS, W == 4 ? 1 : SHORT ? 4 : 2) void k_dw(const uint16_t* xc, int H, const uint16_t* d, int64_t ldd,
                                                        int rows, Tokens tk, OutT* dw, int64_t ld_dw, int accumulate) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int TILE = tile_side(W), WAVE = 32 * W;
  const int cols = tk.columns();
  const float scale = *tk.scale;
  int pm, pn;
  // SHORT: few tokens' xc stays in L2 whole, so dw's rows are written from end to end
  // (131072 x 5120, 128 tokens: the whole call 724 us against 785 in groups of 8)
  const int tiles_h = (H + TILE - 1) / TILE;
  tile_place(blockIdx.x, tiles_h, (rows + TILE - 1) / TILE, pm, pn, SHORT ? tiles_h : 8);
  const int m0 = pm * TILE, n0 = pn * TILE;
  const int K = (cols + 127) / 128 * 128;
  floatx16 acc[W][W];
  // SHORT: one LDS buffer, four workgroups per CU
  if (SHORT || K > 0) {
    const TileOperand ox{xc + m0, (uint32_t)H, H - m0, K};
    const TileOperand od{d + (int64_t)n0 * ldd, (uint32_t)ldd, rows - n0, K};
    if constexpr (SHORT)
      tile_product_short<W, true, false>(ox, od, (cols + TILE_K - 1) / TILE_K, lds, acc);
    else
      tile_product<W, true, false, true>(ox, od, K, 0, K / TILE_K, lds, acc);
  } else {
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int j = 0; j < W; j++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < W; j++)
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = wm * WAVE + 32 * i + 8 * q + 4 * h, n = wn * WAVE + 32 * j + lr;
        const bool in = n0 + n < rows && m0 + m < H;  // H is a multiple of 8
        OutT* out = dw + (int64_t)(n0 + n) * ld_dw + m0 + m;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = acc[i][j][4 * q + r] * scale;
        if constexpr (sizeof(OutT) == 4) {
          if (!in) continue;
          float4* o = reinterpret_cast<float4*>(out);
          float4 s = make_float4(v[0], v[1], v[2], v[3]);
          if (accumulate) {
            const float4 old = *o;
            s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
          }
          store16<STREAM>(o, __builtin_bit_cast(u32x4_t, s));
        } else {
          if (accumulate && in) {
            const u32x2_t old = *reinterpret_cast<const u32x2_t*>(out);
            v[0] += bf16lo(old[0]);
            v[1] += bf16hi(old[0]);
            v[2] += bf16lo(old[1]);
            v[3] += bf16hi(old[1]);
          }
          tile_put<W>(lds, n, m >> 3, h, bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3]));
        }
      }
  if constexpr (sizeof(OutT) == 2) {
    __syncthreads();
    for (int e = threadIdx.x; e < TILE * 8 * W; e += TILE_THREADS) {
      const int n = e / (8 * W), g = e % (8 * W);
      if (n0 + n < rows && m0 + 8 * g < H)
        store16<STREAM>(dw + (int64_t)(n0 + n) * ld_dw + m0 + 8 * g, tile_get<W>(lds, n, g));
    }
  }
}

// How the dx product of n columns of d^T is spread over `units` workgroups: its
// K (the vocabulary rows, `pairs` of 128 of them in a piece) is split into as many
// parts as the units allow, each at least 256 rows deep.  Part p's sums are
// rows p * rows .. of the workspace, FP32.
struct DxSplit {
  int tiles, parts;
  int64_t rows;
  __device__ DxSplit(int n, int side, int tiles_h, int units, int pairs)
      : tiles((n + side - 1) / side), rows((int64_t)tiles * side) {
    parts = max(1, min(units / max(tiles * tiles_h, 1), pairs / 2));
  }
};

// sum[part][i][h] (+)= sum over the part's vocabulary rows of d^T[v][i] w[v][h];
// `rows` vocabulary rows in this piece, `piece` in the largest.
template <int W, bool ONCE>
__global__ __launch_bounds__(TILE_THREADS, W == 4 ? 1 : 2) void k_dx_sum(const uint16_t* w, uint32_t ld_w, int H,
                                                                         const uint16_t* d, int64_t ldd, int rows,
                                                                         int piece, Tokens tk, float* sum,
                                                                         int accumulate) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int TILE = tile_side(W), WAVE = 32 * W;
  const int n_tok = *tk.n, cols = tk.columns();
  const bool two = tk.two();
  const int tiles_h = (H + TILE - 1) / TILE;
  const DxSplit sp(cols, TILE, tiles_h, gridDim.x, (piece + 127) / 128);
  if ((int)blockIdx.x >= tiles_h * sp.tiles * sp.parts) return;
  int pm, pn;
  tile_place(blockIdx.x, tiles_h, sp.tiles * sp.parts, pm, pn);
  const int part = pn / sp.tiles;
  const int m0 = pm * TILE, n0 = (pn - part * sp.tiles) * TILE;
  const int pairs = (rows + 127) / 128;
  const int kt0 = (int)((int64_t)pairs * part / sp.parts) * 2, kt1 = (int)((int64_t)pairs * (part + 1) / sp.parts) * 2;
  if (kt0 == kt1) return;  // in a last piece that is shorter: nothing to add
  floatx16 acc[W][W];
  tile_product<W, true, true, true>(TileOperand{w + m0, ld_w, H - m0, rows, ONCE},
                              TileOperand{d + n0, (uint32_t)ldd, (int)(ldd - n0), pairs * 128}, pairs * 128, kt0, kt1, lds,
                              acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  float* out = sum + part * sp.rows * H;
#pragma unroll
  for (int j = 0; j < W; j++)
#pragma unroll
    for (int i = 0; i < W; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = m0 + wm * WAVE + 32 * i + 8 * q + 4 * h, n = n0 + wn * WAVE + 32 * j + lr;
        if (n >= cols || m >= H || (two && n >= n_tok && n < tk.half)) continue;
        float4* o = reinterpret_cast<float4*>(out + (int64_t)n * H + m);
        float4 s = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        if (accumulate) {
          const float4 old = *o;
          s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
        }
        *o = s;
        if (q == 3) __builtin_amdgcn_sched_barrier(0);  // few old values at a time beside 256 accumulators
      }
}

// dx (BF16) from its FP32 sums, added in order (the smaller part of d last); 0 for
// ignored tokens.  A workgroup takes 1024 / S columns of a token, S slices of its
// parts at a time: S = 8 for many parts (5 tokens, H = 152, 256 parts: 7 us against
// 26), 1 for few (248 tokens, H = 4416: 6 us against 15).
template <int S>
__global__ __launch_bounds__(256) void k_dx(const float* sum, int units, int side, int pairs, int H, Tokens tk,
                                            uint16_t* dx, int64_t ld) {
  __shared__ float4 slices[S == 1 ? 1 : S][S == 1 ? 1 : 256 / S];
  const int64_t t = blockIdx.x;
  const int64_t i = tk.place[t];
  const DxSplit sp(tk.columns(), side, (H + side - 1) / side, units, pairs);
  const int lane = threadIdx.x % (256 / S), slice = threadIdx.x / (256 / S);
  const int c = (blockIdx.y * (256 / S) + lane) * 4;
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (i >= 0 && c < H) {
    const int64_t step = sp.rows * H / 4;
    const int p0 = sp.parts * slice / S, p1 = sp.parts * (slice + 1) / S;
    auto add = [&](int64_t row) {
      const float4* p = reinterpret_cast<const float4*>(sum + row * H + c);
#pragma unroll 8
      for (int q = p0; q < p1; q++) {
        const float4 v = p[q * step];
        f.x += v.x, f.y += v.y, f.z += v.z, f.w += v.w;
      }
    };
    add(i);
    if (tk.two()) add(tk.half + i);
  }
  if constexpr (S > 1) {
    slices[slice][lane] = f;
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int q = 1; q < S; q++) {
      const float4 v = slices[q][lane];
      f.x += v.x, f.y += v.y, f.z += v.z, f.w += v.w;
    }
  }
  if (c >= H) return;
  if (i >= 0) {
    const float scale = *tk.scale;
    f.x *= scale, f.y *= scale, f.z *= scale, f.w *= scale;
  }
  *reinterpret_cast<u32x2_t*>(dx + t * ld + c) = u32x2_t{bf16_pack(f.x, f.y), bf16_pack(f.z, f.w)};
}

__global__ __launch_bounds__(256) void k_zero(void* p, int64_t row_bytes, int64_t ld_bytes) {
  uint8_t* r = static_cast<uint8_t*>(p) + (int64_t)blockIdx.x * ld_bytes;
  for (int64_t c = threadIdx.x * 16; c < row_bytes; c += 256 * 16)
    *reinterpret_cast<u32x4_t*>(r + c) = u32x4_t{0, 0, 0, 0};
}

int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

// Vocabulary rows per backward piece: d of a piece takes up to 512 MiB.
constexpr int64_t kPieceBytes = int64_t(512) << 20;
int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }
int64_t tiles_of(int64_t n, int W) { return (n + tile_side(W) - 1) / tile_side(W); }
int64_t piece_rows(int64_t T, int64_t V) {
  const int64_t r = std::max<int64_t>(kPieceBytes / (2 * up128(T)) / 256 * 256, 256);
  return std::min(r, V);
}

// Tile size of an M x N product with K values of k: the one whose rounds of
// workgroups over a 256-CU MI355X (one large tile per CU, two small ones) take
// less.  Measured (H = 5120 and 2048, V = 10000 .. 131072, T = 64 .. 1000): a round
// of large tiles takes 1.55 us a stage and 10 us around them, one of small tiles
// 1.05 and 4, or 0.75 a stage where each has its CU to itself; of 64 x 64 tiles four
// take 0.7 and 4, two 0.5 and 3.
double round_us(int64_t tiles, double stages, int W) {
  if (W == 4) return (double)((tiles + 255) / 256) * (stages * 1.55 + 10.0);
  if (W == 1) {
    const int64_t rest = tiles % 1024;
    return (double)(tiles / 1024) * (stages * 0.7 + 4.0) +
           (rest == 0 ? 0.0 : rest <= 512 ? stages * 0.5 + 3.0 : stages * 0.7 + 4.0);
  }
  const int64_t rest = tiles % 512;
  return (double)(tiles / 512) * (stages * 1.05 + 4.0) +
         (rest == 0 ? 0.0 : stages * (rest <= 256 ? 0.75 : 1.05) + 4.0);
}
int tile_w(int64_t M, int64_t N, int64_t K) {
  const double stages = (double)((K + TILE_K - 1) / TILE_K);
  const double large = round_us(tiles_of(M, 4) * tiles_of(N, 4), stages, 4);
  return large <= round_us(tiles_of(M, 2) * tiles_of(N, 2), stages, 2) ? 4 : 2;
}
// The same with 64 x 64 tiles, four to a CU: they leave fewer CUs idle and waste less
// on a few tokens, but read LDS twice as often per product (MI355X, forward: 69 x 14757
// x 3160 32 us against 46 with 128 x 128, 496 x 4707 x 4416 40 against 53; 257 x
// 49999 x 2048 97 against 85).
int logits_w(int64_t M, int64_t N, int64_t K) {
  const double stages = (double)((K + TILE_K - 1) / TILE_K);
  const int w = tile_w(M, N, K);
  return round_us(tiles_of(M, 1) * tiles_of(N, 1), stages, 1) < round_us(tiles_of(M, w) * tiles_of(N, w), stages, w) ? 1
                                                                                                                     : w;
}

// Up to here the dw product has few enough stages that four small tiles per CU,
// each unpipelined, beat one large tile, where there are that many (131072 x 5120, d
// and dw: 0.86 against 0.97 ms at 256 tokens, 1.91 against 1.85 at 600, 2.77 against
// 2.53 at 1000; 30000 x 2048: 0.089 against 0.103 at 256, level at 1000).
constexpr int64_t SHORT_DW_TOKENS = 512;

// Workgroups of the dx product: its tiles are as few as T x H gives, so K (a
// piece's vocabulary rows) is split, by the rounds that cost least.
struct DxPlan {
  int W;
  int64_t units;
};
DxPlan dx_plan(int64_t T, int64_t H, int64_t piece) {
  const int64_t stages = (piece + TILE_K - 1) / TILE_K;
  DxPlan best{4, 0};
  double best_us = 1e30;
  for (int W = 4; W >= 2; W -= 2) {
    const int64_t slots = W == 4 ? 256 : 512, tiles = tiles_of(T, W) * tiles_of(H, W);
    for (int64_t r = 1; r <= 4 || r * slots < 2 * tiles + slots; r++) {
      const int64_t parts = std::max<int64_t>(1, std::min(r * slots / tiles, stages / 4));
      // the products, and the parts' FP32 sums, written and read at 4.5 TB/s
      const double us = round_us(tiles * parts, (double)stages / parts, W) +
                        (double)(parts * tiles_of(T, W) * tile_side(W) * H) * 8.0 / 4.5e6;
      if (us < best_us * 0.97) {
        best_us = us;
        best = DxPlan{W, std::max(r * slots, tiles)};
      }
    }
  }
  return best;
}

// The backward workspace: offsets of its parts.
struct BackPlan {
  int64_t piece, ldd;
  DxPlan dxp;
  int64_t d, xc, sum, tok, end;
};
BackPlan back_plan(int64_t T, int64_t V, int64_t H) {
  BackPlan p;
  p.piece = piece_rows(T, V);
  p.ldd = T <= 16 ? 32 : T <= 32 ? 64 : up128(T);  // up to 64 tokens have two columns each
  p.dxp = dx_plan(T, H, p.piece);
  p.d = 0;
  p.xc = up16(up128(p.piece) * p.ldd * 2);
  p.sum = p.xc + up16(up128(T) * H * 2);
  p.tok = p.sum + up16(p.dxp.units * tile_side(p.dxp.W) * tile_side(p.dxp.W) * 4);
  p.end = p.tok + up16((2 * T + 2) * 4);
  return p;
}

// Whether a weight that one tile of tokens reads passes the caches by: one that they
// do not hold, in rows of whole 128-byte lines (others' lines serve two stages: 3 x
// 55044 x 3568 86 us through the caches, 101 past them).
bool passes_once(const void* w, int64_t ld_w, int64_t V, int64_t H) {
  return V * H * 2 >= kStreamBytes && ld_w % 64 == 0 && reinterpret_cast<uintptr_t>(w) % 128 == 0;
}

// Dynamic LDS of a tile kernel: its stages and the token values of a tile.
constexpr int lds_of(int W) { return tile_lds(W) + 3 * tile_side(W) * 4; }
hipError_t allow_lds() {  // beyond 64 KB a kernel has to be told
  static std::atomic<uint64_t> done{0};
  return once_per_device(done, [] {
    hipError_t err = hipSuccess;
    auto allow = [&err](const void* f, int W) {
      if (err == hipSuccess) err = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds_of(W));
    };
    allow(reinterpret_cast<const void*>(&k_logits_stats<4, true, false>), 4);
    allow(reinterpret_cast<const void*>(&k_logits_stats<4, false, false>), 4);
    allow(reinterpret_cast<const void*>(&k_logits_stats<2, true, false>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_stats<2, false, false>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_stats<2, true, true>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_stats<2, false, true>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_grad<4, true, false>), 4);
    allow(reinterpret_cast<const void*>(&k_logits_grad<4, false, false>), 4);
    allow(reinterpret_cast<const void*>(&k_logits_grad<2, true, false>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_grad<2, false, false>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_grad<2, true, true>), 2);
    allow(reinterpret_cast<const void*>(&k_logits_grad<2, false, true>), 2);
    allow(reinterpret_cast<const void*>(&k_dw<4, false, false, uint16_t>), 4);
    allow(reinterpret_cast<const void*>(&k_dw<4, false, false, float>), 4);
    allow(reinterpret_cast<const void*>(&k_dw<4, false, true, uint16_t>), 4);
    allow(reinterpret_cast<const void*>(&k_dw<4, false, true, float>), 4);
    allow(reinterpret_cast<const void*>(&k_dw<2, false, false, uint16_t>), 2);
    allow(reinterpret_cast<const void*>(&k_dw<2, false, false, float>), 2);
    allow(reinterpret_cast<const void*>(&k_dx_sum<4, false>), 4);
    allow(reinterpret_cast<const void*>(&k_dx_sum<2, false>), 2);
    allow(reinterpret_cast<const void*>(&k_dx_sum<2, true>), 2);
    return err;
  });
}

// f(W, EVEN) with the tile size, and whether K is a whole number of pairs of
// stages, as constants
template <typename F>
hipError_t with_tile(int W, bool even, F&& f) {
  using std::integral_constant;
  if (W == 4)
    even ? f(integral_constant<int, 4>{}, std::true_type{}) : f(integral_constant<int, 4>{}, std::false_type{});
  else
    even ? f(integral_constant<int, 2>{}, std::true_type{}) : f(integral_constant<int, 2>{}, std::false_type{});
  return hipGetLastError();
}
// The same with 64 x 64 tiles too.
template <typename F>
hipError_t with_logits_tile(int W, bool even, F&& f) {
  if (W > 1) return with_tile(W, even, f);
  using std::integral_constant;
  even ? f(integral_constant<int, 1>{}, std::true_type{}) : f(integral_constant<int, 1>{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace

int64_t linear_ce_workspace(int64_t T, int64_t V, int64_t H, bool train) {
  const int64_t fwd = up16(tiles_of(V, logits_w(V, T, H)) * T * 8) + up16(T * 4);
  return train ? std::max(fwd, back_plan(T, V, H).end) : fwd;
}

hipError_t launch_linear_ce(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                            const int64_t* labels, float* loss, float* lse, void* workspace, hipStream_t s) {
  if (T == 0) return hipSuccess;
  hipError_t e = allow_lds();
  if (e != hipSuccess) return e;
  const int w_tile = logits_w(V, T, H);
  const int64_t tiles = tiles_of(V, w_tile);
  float2* stats = static_cast<float2*>(workspace);
  float* zlab = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up16(tiles * T * 8));
  const bool once = passes_once(w, ld_w, V, H);
  e = with_logits_tile(w_tile, H % 128 == 0, [&](auto W, auto even) {
    auto* kernel = &k_logits_stats<W.value, even.value, false>;
    if constexpr (W.value < 4)
      if (once && tiles_of(T, W.value) == 1) kernel = &k_logits_stats<W.value, even.value, true>;
    kernel<<<(unsigned)(tiles * tiles_of(T, W.value)), TILE_THREADS, lds_of(W.value), s>>>(
        static_cast<const uint16_t*>(w), (uint32_t)ld_w, (int)V, static_cast<const uint16_t*>(x), (uint32_t)ld_x, (int)T,
        (int)H, labels, stats, zlab);
  });
  if (e != hipSuccess) return e;
  k_loss<<<(unsigned)T, 256, 0, s>>>(stats, (int)tiles, (int)V, labels, zlab, loss, lse);
  return hipGetLastError();
}

hipError_t launch_linear_ce_back(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w,
                                 int64_t ld_w, const int64_t* labels, const float* lse, const float* dloss, void* dx,
                                 int64_t ld_dx, void* dw, int dw_dt, int64_t ld_dw, int accumulate, void* workspace,
                                 hipStream_t s) {
  if (T == 0) {
    if (dw == nullptr || accumulate) return hipSuccess;
    const int64_t es = dw_dt == 0 ? 2 : 4;
    k_zero<<<(unsigned)V, 256, 0, s>>>(dw, H * es, ld_dw * es);
    return hipGetLastError();
  }
  hipError_t e = allow_lds();
  if (e != hipSuccess) return e;
  const BackPlan pl = back_plan(T, V, H);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* d = reinterpret_cast<uint16_t*>(ws + pl.d);  // d^T
  uint16_t* xc = reinterpret_cast<uint16_t*>(ws + pl.xc);
  float* sum = reinterpret_cast<float*>(ws + pl.sum);
  int* tok = reinterpret_cast<int*>(ws + pl.tok);
  const Tokens tk{tok, reinterpret_cast<float*>(tok + 1), tok + 2, tok + 2 + T, T <= 16 ? 16 : T <= 32 ? 32 : 64};
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  if (T <= FEW_LABELS) {
    k_tokens_gather<<<(unsigned)(up128(T) / 4), 256, 0, s>>>(labels, dloss, (int)T, V, xp, ld_x, H, tk, xc);
  } else {
    k_tokens<<<1, 1024, 0, s>>>(labels, dloss, T, V, tk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    k_gather<<<(unsigned)up128(T), 256, 0, s>>>(xp, ld_x, H, tk, xc);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  // a gradient that the caches do not hold
  const bool once = passes_once(w, ld_w, V, H), stream = V * H * (dw_dt == 0 ? 2 : 4) >= kStreamBytes;
  for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
    const int64_t n = std::min(pl.piece, V - v0);
    const uint16_t* wp = static_cast<const uint16_t*>(w) + v0 * ld_w;
    e = with_logits_tile(logits_w(T, n, H), H % 128 == 0, [&](auto W, auto even) {
      // up to 64 tokens are all in the first tile, in two parts
      const int64_t tt = T <= 64 ? 1 : tiles_of(up128(T), W.value), tv = tiles_of(up128(n), W.value);
      auto* kernel = &k_logits_grad<W.value, even.value, false>;
      if constexpr (W.value < 4)
        if (once && tiles_of(T, W.value) == 1) kernel = &k_logits_grad<W.value, even.value, true>;
      kernel<<<(unsigned)(tt * tv), TILE_THREADS, lds_of(W.value), s>>>(
          wp, (uint32_t)ld_w, (int)n, xc, (int)H, (int)tt, v0, tk, labels, lse, dloss, d, pl.ldd);
    });
    if (e != hipSuccess) return e;
    if (dw != nullptr) {
      uint8_t* out = static_cast<uint8_t*>(dw) + v0 * ld_dw * (dw_dt == 0 ? 2 : 4);
      if (T <= FEW_DW_TOKENS) {
        // past the caches in whole 128-byte lines only (2 x 116087 x 1720: 248 us for d and dw, 283 past them)
        const bool lines = ld_dw * (dw_dt == 0 ? 2 : 4) % 128 == 0 && reinterpret_cast<uintptr_t>(dw) % 128 == 0;
        e = few_dw(xc, H, d, pl.ldd, n, T, tk, out, dw_dt, ld_dw, accumulate, stream && lines, s);
      } else {
        auto go = [&](auto W, auto with_short) {
          constexpr bool SHORT = with_short.value;
          const unsigned grid = (unsigned)(tiles_of(H, W.value) * tiles_of(n, W.value));
          const int lds = SHORT ? tile_lds(W.value) / 2 : lds_of(W.value);
          auto run = [&](auto* o) {
            using OutT = std::remove_pointer_t<decltype(o)>;
            auto* kernel = &k_dw<W.value, SHORT, false, OutT>;
            if constexpr (W.value == 4 || SHORT)
              if (stream) kernel = &k_dw<W.value, SHORT, true, OutT>;
            kernel<<<grid, TILE_THREADS, lds, s>>>(xc, (int)H, d, pl.ldd, (int)n, tk, o, ld_dw, accumulate);
          };
          if (dw_dt == 0)
            run(reinterpret_cast<uint16_t*>(out));
          else
            run(reinterpret_cast<float*>(out));
          return hipGetLastError();
        };
        using std::integral_constant;
        if (T <= SHORT_DW_TOKENS && tiles_of(H, 2) * tiles_of(n, 2) > 512)
          e = go(integral_constant<int, 2>{}, std::true_type{});
        else if (tile_w(H, n, T) == 2)
          e = go(integral_constant<int, 2>{}, std::false_type{});
        else
          e = go(integral_constant<int, 4>{}, std::false_type{});
      }
      if (e != hipSuccess) return e;
    }
    if (dx != nullptr) {
      e = with_tile(pl.dxp.W, true, [&](auto W, auto) {
        auto* kernel = &k_dx_sum<W.value, false>;
        if constexpr (W.value < 4)
          if (once && tiles_of(T, W.value) == 1) kernel = &k_dx_sum<W.value, true>;
        kernel<<<(unsigned)pl.dxp.units, TILE_THREADS, lds_of(W.value), s>>>(
            wp, (uint32_t)ld_w, (int)H, d, pl.ldd, (int)n, (int)pl.piece, tk, sum, v0 > 0 ? 1 : 0);
      });
      if (e != hipSuccess) return e;
    }
  }
  if (dx == nullptr) return hipSuccess;
  auto join = [&](auto S) {
    k_dx<S.value><<<dim3((unsigned)T, (unsigned)((H * S.value + 1023) / 1024)), 256, 0, s>>>(
        sum, (int)pl.dxp.units, tile_side(pl.dxp.W), (int)((pl.piece + 127) / 128), (int)H, tk,
        static_cast<uint16_t*>(dx), ld_dx);
  };
  if (pl.dxp.units >= 16 * tiles_of(T, pl.dxp.W) * tiles_of(H, pl.dxp.W))  // 16 parts or more
    join(std::integral_constant<int, 8>{});
  else
    join(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

}  // namespace nvfp4
