// Softmax cross entropy of a linear head and its gradient
// (nvfp4_linear_cross_entropy, nvfp4_linear_cross_entropy_backward), gfx950.
//
// Forward: the logits z = x W^T are formed in 256 x 256 tiles on the BF16 matrix
// cores (bf16_tile.hpp); each tile leaves one (maximum, sum of exp(z - maximum))
// pair per token, and the label's logit; a second kernel joins a token's pairs.
// Backward, on the tokens that have a label only, over pieces of the vocabulary:
// the logits tile is formed again, d = dloss (exp(z - lse) - [v = label]) is held
// as BF16 for the piece, and two products follow: dW = d^T x (whole per piece)
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

#include <mutex>

namespace nvfp4 {

namespace {

// Row m of the tile of register r of MFMA tile i, without the lane's 4 h.
__device__ __forceinline__ int tile_row(int i, int r) { return 32 * i + 8 * (r >> 2) + (r & 3); }

// stats[t][vt] = the pair of token t and vocabulary tile vt; zlab[t] = the
// logit of t's label.
__global__ __launch_bounds__(TILE_THREADS, 1) void k_logits_stats(const uint16_t* w, uint32_t ld_w, int V,
                                                                  const uint16_t* x, uint32_t ld_x, int T, int H,
                                                                  const int64_t* labels, float2* stats, float* zlab) {
  extern __shared__ __align__(16) uint8_t lds[];
  int pm, pn;
  tile_place(blockIdx.x, (V + TILE - 1) / TILE, (T + TILE - 1) / TILE, pm, pn);
  const int m0 = pm * TILE, n0 = pn * TILE;
  floatx16 acc[4][4];
  tile_product<false, false>(TileOperand{w + (int64_t)m0 * ld_w, ld_w, V - m0, H},
                             TileOperand{x + (int64_t)n0 * ld_x, ld_x, T - n0, H}, H, 0, (H + TILE_K - 1) / TILE_K, lds,
                             acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  const int rows = V - m0 - wm * 128 - 4 * h;  // vocabulary rows from the lane's first
  float2 st[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int t = n0 + wn * 128 + 32 * j + lr;
    if (V - m0 < TILE) {
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int r = 0; r < 16; r++)
          if (tile_row(i, r) >= rows) acc[i][j][r] = -INFINITY;  // adds nothing below
    }
    // the label's row from the lane's first, where it is one of the wave's
    const int64_t label = t < T ? labels[t] : -1;
    const int lab = label >= 0 && label < V ? (int)label - m0 - wm * 128 - 4 * h : -1;
    if (__any(lab >= 0 && lab < 128)) {
      float z = 0.0f;
      bool mine = false;  // rows alternate in fours between the lanes of a column
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int r = 0; r < 16; r++) {
          z = lab == tile_row(i, r) ? acc[i][j][r] : z;
          mine = mine || lab == tile_row(i, r);
        }
      if (mine) zlab[t] = z;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) mx = fmaxf(mx, acc[i][j][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float sh = shift_of(mx);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) s += exp_fast(acc[i][j][r] - sh);
    s += __shfl_xor(s, 32, 64);
    st[j] = make_float2(mx, s);
  }
  // join the two waves of a column, in LDS (the stages are free)
  __syncthreads();
  float2* half = reinterpret_cast<float2*>(lds);
  if (wm == 1 && h == 0)
    for (int j = 0; j < 4; j++) half[wn * 128 + 32 * j + lr] = st[j];
  __syncthreads();
  if (wm == 0 && h == 0)
    for (int j = 0; j < 4; j++) {
      const int t = n0 + wn * 128 + 32 * j + lr;
      if (t < T) stats[(int64_t)t * ((V + TILE - 1) / TILE) + pm] = join(st[j], half[wn * 128 + 32 * j + lr]);
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

// One workgroup: token t's place is the number of labelled tokens before it.
__global__ __launch_bounds__(1024) void k_tokens(const int64_t* labels, int64_t T, int64_t V, Tokens tk) {
  __shared__ int sums[1024];
  const int tid = threadIdx.x;
  const int64_t per = (T + 1023) / 1024, t0 = min(T, tid * per), t1 = min(T, t0 + per);
  int c = 0;
  for (int64_t t = t0; t < t1; t++) c += labels[t] >= 0 && labels[t] < V ? 1 : 0;
  sums[tid] = c;
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
  if (tid == 1023) *tk.n = sums[1023];
}

// xc[i] = x[list[i]] for the n labelled tokens (nothing else of x is read
// again), then zeros up to a multiple of 64 rows (K of the dW product).
__global__ __launch_bounds__(256) void k_gather(const uint16_t* x, int64_t ld_x, int64_t H, Tokens tk, uint16_t* xc) {
  const int64_t i = blockIdx.x;
  const int n = *tk.n;
  if (i >= (n + 63) / 64 * 64) return;
  const uint16_t* src = x + (i < n ? (int64_t)tk.list[i] * ld_x : 0);
  for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8)
    *reinterpret_cast<u32x4_t*>(xc + i * H + c) =
        i < n ? *reinterpret_cast<const u32x4_t*>(src + c) : u32x4_t{0, 0, 0, 0};
}

// ---- a BF16 tile through LDS: rows n of 256 values of m (512 bytes); the
// 16-byte chunk g of row n lies in slot g ^ (n & 31), so that the 32 rows a wave
// writes at once fall into different banks.

// Four consecutive values of m (from 8 g + 4 half) of row n.
__device__ __forceinline__ void tile_put(uint8_t* lds, int n, int g, int half, uint32_t lo, uint32_t hi) {
  *reinterpret_cast<u32x2_t*>(lds + n * 512 + ((g ^ (n & 31)) << 4) + 8 * half) = u32x2_t{lo, hi};
}
__device__ __forceinline__ u32x4_t tile_get(const uint8_t* lds, int n, int g) {
  return *reinterpret_cast<const u32x4_t*>(lds + n * 512 + ((g ^ (n & 31)) << 4));
}

// d^T of a piece of the vocabulary, BF16 [rows up to a multiple of 64][ldd], one
// column per labelled token, zeros in the columns from n up to a multiple of 64
// and in the rows past the piece's last: both are K of a later product.
__global__ __launch_bounds__(TILE_THREADS, 1) void k_logits_grad(const uint16_t* w, uint32_t ld_w, int rows,
                                                                 const uint16_t* xc, int H, int tiles_t, int64_t v_first,
                                                                 Tokens tk, const int64_t* labels, const float* lse,
                                                                 const float* dloss, uint16_t* d, int64_t ldd) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int n_tok = *tk.n;
  int pm, pn;  // token tile, vocabulary tile
  tile_place(blockIdx.x, tiles_t, (rows + TILE - 1) / TILE, pm, pn);
  const int m0 = pm * TILE, n0 = pn * TILE;
  if (m0 >= n_tok) return;
  floatx16 acc[4][4];
  tile_product<false, false>(TileOperand{xc + (int64_t)m0 * H, (uint32_t)H, n_tok - m0, H},
                             TileOperand{w + (int64_t)n0 * ld_w, ld_w, rows - n0, H}, H, 0, (H + TILE_K - 1) / TILE_K, lds,
                             acc);
  // what the tile's tokens hold: lse, dloss, and the label's row in this tile (or -1)
  __syncthreads();
  float* s_lse = reinterpret_cast<float*>(lds + TILE_LDS);
  float* s_g = s_lse + TILE;
  int* s_lab = reinterpret_cast<int*>(s_g + TILE);
  if (threadIdx.x < TILE) {
    const int i = m0 + threadIdx.x;
    float l = 0.0f, g = 0.0f;
    int64_t lab = -1;
    if (i < n_tok) {
      const int t = tk.list[i];
      l = lse[t];
      g = dloss[t];
      lab = labels[t] - v_first - n0;
    }
    s_lse[threadIdx.x] = l;
    s_g[threadIdx.x] = g;
    s_lab[threadIdx.x] = lab >= 0 && lab < TILE ? (int)lab : -1;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  // a label of the wave's 128 tokens among its 128 vocabulary rows?
  const int lab0 = s_lab[wm * 128 + lane] >> 7, lab1 = s_lab[wm * 128 + 64 + lane] >> 7;  // -1 stays -1
  const bool hit = __any(lab0 == wn || lab1 == wn);
  auto put = [&](auto with_labels) {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = wm * 128 + 32 * i + 8 * q + 4 * h;
        const float4 l = *reinterpret_cast<const float4*>(s_lse + m);
        const float4 g = *reinterpret_cast<const float4*>(s_g + m);
        int4 lab = make_int4(-1, -1, -1, -1);
        if constexpr (with_labels.value) lab = *reinterpret_cast<const int4*>(s_lab + m);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int n = wn * 128 + 32 * j + lr;
          float p0 = exp_fast(acc[i][j][4 * q] - l.x), p1 = exp_fast(acc[i][j][4 * q + 1] - l.y);
          float p2 = exp_fast(acc[i][j][4 * q + 2] - l.z), p3 = exp_fast(acc[i][j][4 * q + 3] - l.w);
          if constexpr (with_labels.value) {
            p0 -= lab.x == n ? 1.0f : 0.0f;
            p1 -= lab.y == n ? 1.0f : 0.0f;
            p2 -= lab.z == n ? 1.0f : 0.0f;
            p3 -= lab.w == n ? 1.0f : 0.0f;
          }
          tile_put(lds, n, m >> 3, h, bf16_pack(p0 * g.x, p1 * g.y), bf16_pack(p2 * g.z, p3 * g.w));
        }
        __builtin_amdgcn_sched_barrier(0);  // few token values at a time beside 256 accumulators
      }
  };
  if (hit)
    put(std::true_type{});
  else
    put(std::false_type{});
  __syncthreads();
  const int padded = (rows + 63) / 64 * 64;
  for (int e = threadIdx.x; e < TILE * 32; e += TILE_THREADS) {
    const int n = e >> 5, g = e & 31;
    const int c = m0 + 8 * g;
    if (n0 + n >= padded || c >= ldd) continue;
    u32x4_t v = {0, 0, 0, 0};
    if (n0 + n < rows && c < n_tok) {
      v = tile_get(lds, n, g);
      if (c + 8 > n_tok) {
#pragma unroll
        for (int k = 0; k < 4; k++)
          v[k] &= (c + 2 * k < n_tok ? 0xFFFFu : 0u) | (c + 2 * k + 1 < n_tok ? 0xFFFF0000u : 0u);
      }
    }
    *reinterpret_cast<u32x4_t*>(d + (int64_t)(n0 + n) * ldd + c) = v;
  }
}

// dw[v][h] (+)= sum over the labelled tokens of d^T[v][i] xc[i][h]
template <typename OutT>
__global__ __launch_bounds__(TILE_THREADS, 1) void k_dw(const uint16_t* xc, int H, const uint16_t* d, int64_t ldd,
                                                        int rows, Tokens tk, OutT* dw, int64_t ld_dw, int accumulate) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int n_tok = *tk.n;
  int pm, pn;
  tile_place(blockIdx.x, (H + TILE - 1) / TILE, (rows + TILE - 1) / TILE, pm, pn);
  const int m0 = pm * TILE, n0 = pn * TILE;
  const int K = (n_tok + 63) / 64 * 64;
  floatx16 acc[4][4];
  if (K > 0) {
    tile_product<true, false>(TileOperand{xc + m0, (uint32_t)H, H - m0, K},
                              TileOperand{d + (int64_t)n0 * ldd, (uint32_t)ldd, rows - n0, K}, K, 0, K / TILE_K, lds, acc);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = wm * 128 + 32 * i + 8 * q + 4 * h, n = wn * 128 + 32 * j + lr;
        const bool in = n0 + n < rows && m0 + m < H;  // H is a multiple of 8
        OutT* out = dw + (int64_t)(n0 + n) * ld_dw + m0 + m;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = acc[i][j][4 * q + r];
        if constexpr (sizeof(OutT) == 4) {
          if (!in) continue;
          float4* o = reinterpret_cast<float4*>(out);
          float4 s = make_float4(v[0], v[1], v[2], v[3]);
          if (accumulate) {
            const float4 old = *o;
            s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
          }
          *o = s;
        } else {
          if (accumulate && in) {
            const u32x2_t old = *reinterpret_cast<const u32x2_t*>(out);
            v[0] += bf16lo(old[0]);
            v[1] += bf16hi(old[0]);
            v[2] += bf16lo(old[1]);
            v[3] += bf16hi(old[1]);
          }
          tile_put(lds, n, m >> 3, h, bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3]));
        }
      }
  if constexpr (sizeof(OutT) == 2) {
    __syncthreads();
    for (int e = threadIdx.x; e < TILE * 32; e += TILE_THREADS) {
      const int n = e >> 5, g = e & 31;
      if (n0 + n < rows && m0 + 8 * g < H)
        *reinterpret_cast<u32x4_t*>(dw + (int64_t)(n0 + n) * ld_dw + m0 + 8 * g) = tile_get(lds, n, g);
    }
  }
}

// sum[part][i][h] (+)= sum over the part's vocabulary rows of d^T[v][i] w[v][h]
// (FP32): the piece's rows are split into `parts` contiguous ranges of stages.
__global__ __launch_bounds__(TILE_THREADS, 1) void k_dx_sum(const uint16_t* w, uint32_t ld_w, int H, const uint16_t* d,
                                                            int64_t ldd, int rows, int tiles_t, int parts, Tokens tk,
                                                            float* sum, int64_t T, int accumulate) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int n_tok = *tk.n;
  const int tiles_h = (H + TILE - 1) / TILE;
  int pm, pn;
  tile_place(blockIdx.x, tiles_h, tiles_t * parts, pm, pn);
  const int part = pn / tiles_t;
  const int m0 = pm * TILE, n0 = (pn - part * tiles_t) * TILE;
  if (n0 >= n_tok) return;
  const int KT = (rows + TILE_K - 1) / TILE_K;
  const int kt0 = (int)((int64_t)KT * part / parts), kt1 = (int)((int64_t)KT * (part + 1) / parts);
  if (kt0 == kt1) {  // fewer stages than parts: nothing to add
    if (accumulate) return;
  }
  floatx16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  if (kt0 < kt1)
    tile_product<true, true>(TileOperand{w + m0, ld_w, H - m0, rows},
                             TileOperand{d + n0, (uint32_t)ldd, (int)(ldd - n0), KT * TILE_K}, rows, kt0, kt1, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  float* out = sum + (int64_t)part * T * H;
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int m = m0 + wm * 128 + 32 * i + 8 * q + 4 * h, n = n0 + wn * 128 + 32 * j + lr;
        if (n >= n_tok || m >= H) continue;
        float4* o = reinterpret_cast<float4*>(out + (int64_t)n * H + m);
        float4 s = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        if (accumulate) {
          const float4 old = *o;
          s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
        }
        *o = s;
      }
}

// dx (BF16) from its FP32 sums, added in order; 0 for ignored tokens
__global__ __launch_bounds__(256) void k_dx(const float* sum, int parts, int64_t T, int64_t H, Tokens tk, uint16_t* dx,
                                            int64_t ld) {
  const int64_t t = blockIdx.x;
  const int64_t i = tk.place[t];
  for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8) {
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; q++) f[q] = 0.0f;
    if (i >= 0)
      for (int p = 0; p < parts; p++) {
        const float4* s = reinterpret_cast<const float4*>(sum + (p * T + i) * H + c);
        const float4 a = s[0], b = s[1];
        f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
        f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
      }
    *reinterpret_cast<u32x4_t*>(dx + t * ld + c) = VecOf<uint16_t>::pack(f);
  }
}

__global__ __launch_bounds__(256) void k_zero(void* p, int64_t row_bytes, int64_t ld_bytes) {
  uint8_t* r = static_cast<uint8_t*>(p) + (int64_t)blockIdx.x * ld_bytes;
  for (int64_t c = threadIdx.x * 16; c < row_bytes; c += 256 * 16)
    *reinterpret_cast<u32x4_t*>(r + c) = u32x4_t{0, 0, 0, 0};
}

int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

// Vocabulary rows per backward piece: d of a piece takes up to 512 MiB.
constexpr int64_t kPieceBytes = int64_t(512) << 20;
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }
int64_t tiles_of(int64_t n) { return (n + TILE - 1) / TILE; }
int64_t piece_rows(int64_t T, int64_t V) {
  const int64_t r = std::max<int64_t>(kPieceBytes / (2 * up64(T)) / TILE * TILE, TILE);
  return std::min(r, V);
}

// Parts of the dx product's K (a piece's vocabulary rows): as many as fill the
// compute units of a 256-CU MI355X best, each at least 8 stages deep, at most 16.
int64_t dx_parts(int64_t T, int64_t H, int64_t piece) {
  const int64_t tiles = tiles_of(T) * tiles_of(H), stages = (piece + TILE_K - 1) / TILE_K;
  int64_t best = 1;
  double best_cost = 1e30;
  for (int64_t s = 1; s <= 16 && (s == 1 || stages / s >= 8); s++) {
    // rounds of workgroups times the stages of one, plus the store of its FP32 tile (about 8 stages' time)
    const double cost = (double)((tiles * s + 255) / 256) * ((double)stages / s + 8.0);
    if (cost < best_cost * 0.98) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// The backward workspace: offsets of its parts.
struct BackPlan {
  int64_t piece, ldd, parts;
  int64_t dt, d, xc, sum, tok, end;
};
BackPlan back_plan(int64_t T, int64_t V, int64_t H) {
  BackPlan p;
  p.dt = 0;
  if (T <= FEW_TOKENS) {  // the whole vocabulary at once, d in both orientations
    p.piece = V;
    p.ldd = few_ldt(T);
    p.parts = few_dx_parts(T, V, H);
    p.d = up16(few_rows(V) * p.ldd * 2);
    p.xc = p.d + up16(few_tokens(T) * few_rows(V) * 2);
  } else {
    p.piece = piece_rows(T, V);
    p.ldd = up64(T);
    p.parts = dx_parts(T, H, p.piece);
    p.d = p.xc = up16(up64(p.piece) * p.ldd * 2);
  }
  p.sum = p.xc + up16(up64(T) * H * 2);
  p.tok = p.sum + up16(p.parts * T * H * 4);
  p.end = p.tok + up16((2 * T + 1) * 4);
  return p;
}

// Vocabulary tiles of the forward's pairs.
int64_t stats_tiles(int64_t T, int64_t V) { return T <= FEW_TOKENS ? few_rows(V) / FEW_ROWS : tiles_of(V); }

// Largest dynamic LDS of every tile kernel, set once.
constexpr int kTileLds = TILE_LDS + 3 * TILE * 4;
hipError_t allow_lds() {
  static std::once_flag once;
  static hipError_t err = hipSuccess;
  std::call_once(once, [] {
    const void* fns[] = {reinterpret_cast<const void*>(&k_logits_stats), reinterpret_cast<const void*>(&k_logits_grad),
                         reinterpret_cast<const void*>(&k_dw<uint16_t>), reinterpret_cast<const void*>(&k_dw<float>),
                         reinterpret_cast<const void*>(&k_dx_sum)};
    for (const void* f : fns)
      if (err == hipSuccess) err = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, kTileLds);
  });
  return err;
}

}  // namespace

int64_t linear_ce_workspace(int64_t T, int64_t V, int64_t H, bool train) {
  const int64_t fwd = up16(stats_tiles(T, V) * T * 8) + up16(T * 4);
  return train ? std::max(fwd, back_plan(T, V, H).end) : fwd;
}

hipError_t launch_linear_ce(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                            const int64_t* labels, float* loss, float* lse, void* workspace, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int tiles = (int)stats_tiles(T, V);
  float2* stats = static_cast<float2*>(workspace);
  float* zlab = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up16((int64_t)tiles * T * 8));
  const uint16_t* wp = static_cast<const uint16_t*>(w);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  hipError_t e;
  if (T <= FEW_TOKENS) {
    e = few_stats(wp, (uint32_t)ld_w, V, xp, (uint32_t)ld_x, T, H, labels, stats, zlab, s);
  } else {
    if ((e = allow_lds()) != hipSuccess) return e;
    k_logits_stats<<<(unsigned)(tiles * tiles_of(T)), TILE_THREADS, kTileLds, s>>>(
        wp, (uint32_t)ld_w, (int)V, xp, (uint32_t)ld_x, (int)T, (int)H, labels, stats, zlab);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  k_loss<<<(unsigned)T, 256, 0, s>>>(stats, tiles, (int)V, labels, zlab, loss, lse);
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
  const BackPlan pl = back_plan(T, V, H);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* d = reinterpret_cast<uint16_t*>(ws + pl.dt);  // d^T
  uint16_t* xc = reinterpret_cast<uint16_t*>(ws + pl.xc);
  float* sum = reinterpret_cast<float*>(ws + pl.sum);
  int* tok = reinterpret_cast<int*>(ws + pl.tok);
  const Tokens tk{tok, tok + 1, tok + 1 + T};
  k_tokens<<<1, 1024, 0, s>>>(labels, T, V, tk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_gather<<<(unsigned)up64(T), 256, 0, s>>>(static_cast<const uint16_t*>(x), ld_x, H, tk, xc);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (T <= FEW_TOKENS) {
    uint16_t* dr = reinterpret_cast<uint16_t*>(ws + pl.d);
    const uint16_t* wp = static_cast<const uint16_t*>(w);
    e = few_grad(wp, (uint32_t)ld_w, V, xc, T, H, tk, labels, lse, dloss, d, dr, s);
    if (e == hipSuccess && dw != nullptr)
      e = few_dw(xc, H, d, pl.ldd, V, T, tk, dw, dw_dt, ld_dw, accumulate, s);
    if (e == hipSuccess && dx != nullptr) e = few_dx(wp, (uint32_t)ld_w, V, dr, T, H, tk, sum, s);
    if (e != hipSuccess) return e;
    if (dx != nullptr)
      k_dx<<<(unsigned)T, 256, 0, s>>>(sum, (int)pl.parts, T, H, tk, static_cast<uint16_t*>(dx), ld_dx);
    return hipGetLastError();
  }
  if ((e = allow_lds()) != hipSuccess) return e;
  const int tt = (int)tiles_of(T);
  const int64_t th = tiles_of(H);
  for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
    const int64_t n = std::min(pl.piece, V - v0);
    const int64_t tv = tiles_of(n);
    const uint16_t* wp = static_cast<const uint16_t*>(w) + v0 * ld_w;
    k_logits_grad<<<(unsigned)(tt * tv), TILE_THREADS, kTileLds, s>>>(wp, (uint32_t)ld_w, (int)n, xc, (int)H, tt, v0,
                                                                      tk, labels, lse, dloss, d, pl.ldd);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (dw != nullptr && T <= FEW_DW_TOKENS) {
      void* out = static_cast<uint8_t*>(dw) + v0 * ld_dw * (dw_dt == 0 ? 2 : 4);
      if ((e = few_dw(xc, H, d, pl.ldd, n, T, tk, out, dw_dt, ld_dw, accumulate, s)) != hipSuccess) return e;
    } else if (dw != nullptr) {
      if (dw_dt == 0)
        k_dw<<<(unsigned)(th * tv), TILE_THREADS, kTileLds, s>>>(
            xc, (int)H, d, pl.ldd, (int)n, tk, static_cast<uint16_t*>(dw) + v0 * ld_dw, ld_dw, accumulate);
      else
        k_dw<<<(unsigned)(th * tv), TILE_THREADS, kTileLds, s>>>(xc, (int)H, d, pl.ldd, (int)n, tk,
                                                                 static_cast<float*>(dw) + v0 * ld_dw, ld_dw,
                                                                 accumulate);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (dx != nullptr) {
      k_dx_sum<<<(unsigned)(th * tt * pl.parts), TILE_THREADS, kTileLds, s>>>(
          wp, (uint32_t)ld_w, (int)H, d, pl.ldd, (int)n, tt, (int)pl.parts, tk, sum, T, v0 > 0 ? 1 : 0);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (dx == nullptr) return hipSuccess;
  k_dx<<<(unsigned)T, 256, 0, s>>>(sum, (int)pl.parts, T, H, tk, static_cast<uint16_t*>(dx), ld_dx);
  return hipGetLastError();
}

}  // namespace nvfp4
