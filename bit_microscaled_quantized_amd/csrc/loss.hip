// Softmax cross entropy of a linear head and its gradient
// (nvfp4_linear_cross_entropy, nvfp4_linear_cross_entropy_backward), gfx950.
//
// Forward: the logits z = x W^T are formed in tiles on the BF16 matrix cores;
// each tile leaves one (maximum, sum of exp(z - maximum)) pair per token, and
// the label's logit; a second kernel joins the pairs of a token.
// Backward: over pieces of the vocabulary, the logits tile is formed again,
// d = dloss (exp(z - lse) - [v = label]) is held as BF16 for the piece, and two
// products follow: dW = d^T x (whole per piece) and dx += d W (FP32 in the
// workspace across pieces, rounded to BF16 once at the end).
#include "layers_device.hpp"
#include "layers_launch.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// ---- one 128 x 128 tile of C[m][n] = sum_k A(m, k) B(n, k)
//
// 256 threads = 4 waves in a 2 x 2 grid, wave tile 64 x 64 = 2 x 2 MFMA tiles
// of 32 x 32.  An operand is row-major with K along its rows (KMAJOR false:
// element (m, k) at p[m * ld + k]) or K down its columns (KMAJOR true: at
// p[k * ld + m]); either is staged to LDS as rows of K, zeros past its ends.
constexpr int TM = 128, TN = 128, TK = 32;
constexpr int LDK = TK + 8;  // LDS row of TK elements, padded against bank conflicts

struct Operand {
  const uint16_t* p;
  int64_t ld;
  int64_t rows;  // valid m
};

template <bool KMAJOR>
__device__ __forceinline__ void stage(const Operand& o, int64_t m0, int64_t k0, int64_t K, uint16_t* lds) {
  const int tid = threadIdx.x;
  if constexpr (!KMAJOR) {
    // 128 rows x 4 vectors of 8
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int r = (tid >> 2) + 64 * q, c = (tid & 3) * 8;
      u32x4_t v = {0, 0, 0, 0};
      if (m0 + r < o.rows && k0 + c < K)
        v = load_vec(o.p + (m0 + r) * o.ld + k0 + c, (int)min<int64_t>(8, K - k0 - c));
      *reinterpret_cast<u32x4_t*>(lds + r * LDK + c) = v;
    }
  } else {
    // 32 values of k x 16 vectors of 8 along m, scattered
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int k = (tid >> 4) + 16 * q, m = (tid & 15) * 8;
      u32x4_t v = {0, 0, 0, 0};
      if (k0 + k < K && m0 + m < o.rows)
        v = load_vec(o.p + (k0 + k) * o.ld + m0 + m, (int)min<int64_t>(8, o.rows - m0 - m));
#pragma unroll
      for (int i = 0; i < 8; i++) lds[(m + i) * LDK + k] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// acc[i][j][r]: row wm*64 + 32i + 8(r/4) + 4h + r%4, column wn*64 + 32j + l%32
// of the tile (h = l/32).
template <bool AK, bool BK>
__device__ __forceinline__ void tile_product(const Operand& a, const Operand& b, int64_t m0, int64_t n0, int64_t K,
                                             uint16_t* lds, floatx16 (&acc)[2][2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  uint16_t* la = lds;
  uint16_t* lb = lds + TM * LDK;
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;
  for (int64_t k0 = 0; k0 < K; k0 += TK) {
    __syncthreads();
    stage<AK>(a, m0, k0, K, la);
    stage<BK>(b, n0, k0, K, lb);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < TK / 16; s++) {
      bf16x8_t fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        fa[i] = *reinterpret_cast<const bf16x8_t*>(la + (wm * 64 + 32 * i + lr) * LDK + 16 * s + 8 * h);
        fb[i] = *reinterpret_cast<const bf16x8_t*>(lb + (wn * 64 + 32 * i + lr) * LDK + 16 * s + 8 * h);
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }
}

constexpr int LDS_ELEMS = (TM + TN) * LDK;

// (maximum m, sum of exp(z - m)) of some of a token's logits.  An infinite
// maximum (no logits, only -inf among them, or a +inf) is taken as 0 in the
// exponents, so that the sum is 0, inf or NaN as it is without the shift.
__device__ __forceinline__ float shift_of(float m) { return __builtin_fabsf(m) == INFINITY ? 0.0f : m; }
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float fa = __builtin_fabsf(a.x) == INFINITY ? 1.0f : expf(a.x - m);
  const float fb = __builtin_fabsf(b.x) == INFINITY ? 1.0f : expf(b.x - m);
  return make_float2(m, a.y * fa + b.y * fb);
}

// ---- logits tiles: rows are the vocabulary, columns the tokens, so a lane
// holds 32 logits of each of two tokens.

// stats[vt][t] = (max, sum of exp(z - max)) over the vocabulary tile vt
__global__ __launch_bounds__(256) void k_logits_stats(Operand w, Operand x, int H, const int64_t* labels,
                                                      float2* stats, float* zlab) {
  __shared__ __align__(16) uint16_t lds[LDS_ELEMS];
  __shared__ float2 half[TN];
  floatx16 acc[2][2];
  const int64_t m0 = (int64_t)blockIdx.x * TM, n0 = (int64_t)blockIdx.y * TN;
  tile_product<false, false>(w, x, m0, n0, H, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
  float2 st[2];
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int64_t t = n0 + wn * 64 + 32 * j + lr;
    const int64_t lab = t < x.rows ? labels[t] : -1;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int64_t v = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
        if (v >= w.rows) continue;
        mx = fmaxf(mx, acc[i][j][r]);
        if (v == lab) zlab[t] = acc[i][j][r];
      }
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float sh = shift_of(mx);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int64_t v = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
        if (v < w.rows) s += expf(acc[i][j][r] - sh);
      }
    s += __shfl_xor(s, 32, 64);
    st[j] = make_float2(mx, s);
  }
  // join the two waves of a column
  if (wm == 1 && h == 0)
    for (int j = 0; j < 2; j++) half[wn * 64 + 32 * j + lr] = st[j];
  __syncthreads();
  if (wm == 0 && h == 0)
    for (int j = 0; j < 2; j++) {
      const int64_t t = n0 + wn * 64 + 32 * j + lr;
      if (t < x.rows)
        stats[(int64_t)blockIdx.x * x.rows + t] = join(st[j], half[wn * 64 + 32 * j + lr]);
    }
}

// lse and loss of a token from its `tiles` pairs: 64 tokens per workgroup,
// four slices of tiles each.
__global__ __launch_bounds__(256) void k_loss(const float2* stats, int tiles, int64_t T, int64_t V,
                                              const int64_t* labels, const float* zlab, float* loss, float* lse) {
  __shared__ float2 part[4][64];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 64 + lane;
  float2 st = make_float2(-INFINITY, 0.0f);
  if (t < T)
    for (int q = tiles * slice / 4; q < tiles * (slice + 1) / 4; q++) st = join(st, stats[(int64_t)q * T + t]);
  part[slice][lane] = st;
  __syncthreads();
  if (slice != 0 || t >= T) return;
  for (int q = 1; q < 4; q++) st = join(st, part[q][lane]);
  const float l = st.x + logf(st.y);
  lse[t] = l;
  const int64_t lab = labels[t];
  loss[t] = lab >= 0 && lab < V ? l - zlab[t] : 0.0f;
}

// ---- backward: the tokens that have a label come first

// What the backward pass knows of its n[0] labelled tokens, in order: their
// labels, lse, dloss, and of every token its place among them (or -1).
struct Tokens {
  int* n;
  int* place;
  int* list;
};

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

// xc[i] = x[list[i]] for the labelled tokens (nothing else of x is read again)
__global__ __launch_bounds__(256) void k_gather(const uint16_t* x, int64_t ld_x, int64_t H, Tokens tk, uint16_t* xc) {
  const int64_t i = blockIdx.x;
  if (i >= *tk.n) return;
  const uint16_t* src = x + (int64_t)tk.list[i] * ld_x;
  for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8)
    *reinterpret_cast<u32x4_t*>(xc + i * H + c) = *reinterpret_cast<const u32x4_t*>(src + c);
}

// d^T of a piece of the vocabulary, BF16 [piece][ldd], one column per labelled token
__global__ __launch_bounds__(256) void k_logits_grad(Operand w, Operand x, int H, int64_t v_first, Tokens tk,
                                                     const int64_t* labels, const float* lse, const float* dloss,
                                                     uint16_t* d, int64_t ldd) {
  __shared__ __align__(16) uint16_t lds[LDS_ELEMS];
  floatx16 acc[2][2];
  const int64_t m0 = (int64_t)blockIdx.x * TM, n0 = (int64_t)blockIdx.y * TN;
  x.rows = *tk.n;
  if (n0 >= x.rows) return;
  tile_product<false, false>(w, x, m0, n0, H, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const int64_t i0 = n0 + wn * 64 + 32 * j + lr;
    if (i0 >= x.rows) continue;
    const int t = tk.list[i0];
    const int64_t lab = labels[t];
    const float l = lse[t], g = dloss[t];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int64_t m = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
        if (m >= w.rows) continue;
        const float p = expf(acc[i][j][r] - l) - (v_first + m == lab ? 1.0f : 0.0f);
        d[m * ldd + i0] = (uint16_t)bf16_pack(g * p, 0.0f);
      }
  }
}

// C (+)= A . B; FP32 or BF16 output.  The number of labelled tokens is A's
// rows (NROWS) or K.
template <bool AK, bool BK, bool NROWS, typename OutT>
__global__ __launch_bounds__(256) void k_product(Operand a, Operand b, int64_t K, const int* n_tok, OutT* c,
                                                 int64_t ldc, int accumulate) {
  __shared__ __align__(16) uint16_t lds[LDS_ELEMS];
  floatx16 acc[2][2];
  const int64_t m0 = (int64_t)blockIdx.x * TM, n0 = (int64_t)blockIdx.y * TN;
  if constexpr (NROWS) {
    a.rows = *n_tok;
    if (m0 >= a.rows) return;
  } else {
    K = *n_tok;
  }
  tile_product<AK, BK>(a, b, m0, n0, K, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, h = lane >> 5, lr = lane & 31;
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int64_t m = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
        const int64_t n = n0 + wn * 64 + 32 * j + lr;
        if (m >= a.rows || n >= b.rows) continue;
        float v = acc[i][j][r];
        OutT* p = c + m * ldc + n;
        if (accumulate) v += VecOf<OutT>::one(p);
        if constexpr (sizeof(OutT) == 4)
          *p = v;
        else
          *p = (uint16_t)bf16_pack(v, 0.0f);
      }
}

// dx (BF16) from its FP32 sum, 0 for ignored tokens
__global__ __launch_bounds__(256) void k_dx(const float* sum, int64_t H, Tokens tk, uint16_t* dx, int64_t ld) {
  const int64_t t = blockIdx.x;
  const int64_t i = tk.place[t];
  for (int64_t c = threadIdx.x * 8; c < H; c += 256 * 8) {
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; q++) f[q] = i >= 0 ? sum[i * H + c + q] : 0.0f;
    *reinterpret_cast<u32x4_t*>(dx + t * ld + c) = VecOf<uint16_t>::pack(f);
  }
}

__global__ __launch_bounds__(256) void k_zero(void* p, int64_t rows, int64_t row_bytes, int64_t ld_bytes) {
  uint8_t* r = static_cast<uint8_t*>(p) + (int64_t)blockIdx.x * ld_bytes;
  for (int64_t c = threadIdx.x * 16; c < row_bytes; c += 256 * 16)
    *reinterpret_cast<u32x4_t*>(r + c) = u32x4_t{0, 0, 0, 0};
}

int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }

// Vocabulary rows per backward piece: d of a piece takes up to 512 MiB.
constexpr int64_t kPieceBytes = int64_t(512) << 20;
int64_t piece_rows(int64_t T, int64_t V) {
  const int64_t ldd = (T + 7) / 8 * 8;
  const int64_t r = std::max<int64_t>(kPieceBytes / (2 * ldd) / TM * TM, TM);
  return std::min(r, V);
}

// The backward workspace: bytes of each part, from its start.
struct BackPlan {
  int64_t piece, ldd;           // vocabulary rows per piece, tokens padded to 8
  int64_t d, xc, sum, tok, end;  // offsets
};
BackPlan back_plan(int64_t T, int64_t V, int64_t H) {
  BackPlan p;
  p.piece = piece_rows(T, V);
  p.ldd = (T + 7) / 8 * 8;
  p.d = 0;
  p.xc = p.d + up16(p.piece * p.ldd * 2);
  p.sum = p.xc + up16(T * H * 2);
  p.tok = p.sum + up16(T * H * 4);
  p.end = p.tok + up16((2 * T + 1) * 4);
  return p;
}

}  // namespace

int64_t linear_ce_workspace(int64_t T, int64_t V, int64_t H, bool train) {
  const int64_t fwd = up16((V + TM - 1) / TM * T * 8) + up16(T * 4);
  if (!train) return fwd;
  const int64_t bwd = back_plan(T, V, H).end;
  return std::max(fwd, bwd);
}

hipError_t launch_linear_ce(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w, int64_t ld_w,
                            const int64_t* labels, float* loss, float* lse, void* workspace, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int tiles = (int)((V + TM - 1) / TM);
  float2* stats = static_cast<float2*>(workspace);
  float* zlab = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up16((int64_t)tiles * T * 8));
  const Operand ow{static_cast<const uint16_t*>(w), ld_w, V}, ox{static_cast<const uint16_t*>(x), ld_x, T};
  k_logits_stats<<<dim3(tiles, (unsigned)((T + TN - 1) / TN)), 256, 0, s>>>(ow, ox, (int)H, labels, stats, zlab);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_loss<<<(unsigned)((T + 63) / 64), 256, 0, s>>>(stats, tiles, T, V, labels, zlab, loss, lse);
  return hipGetLastError();
}

hipError_t launch_linear_ce_back(int64_t T, int64_t V, int64_t H, const void* x, int64_t ld_x, const void* w,
                                 int64_t ld_w, const int64_t* labels, const float* lse, const float* dloss, void* dx,
                                 int64_t ld_dx, void* dw, int dw_dt, int64_t ld_dw, int accumulate, void* workspace,
                                 hipStream_t s) {
  if (T == 0) {
    if (dw == nullptr || accumulate) return hipSuccess;
    const int64_t es = dw_dt == 0 ? 2 : 4;
    k_zero<<<(unsigned)V, 256, 0, s>>>(dw, V, H * es, ld_dw * es);
    return hipGetLastError();
  }
  const BackPlan pl = back_plan(T, V, H);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* d = reinterpret_cast<uint16_t*>(ws + pl.d);
  uint16_t* xc = reinterpret_cast<uint16_t*>(ws + pl.xc);
  float* sum = reinterpret_cast<float*>(ws + pl.sum);
  int* tok = reinterpret_cast<int*>(ws + pl.tok);
  const Tokens tk{tok, tok + 1, tok + 1 + T};
  k_tokens<<<1, 1024, 0, s>>>(labels, T, V, tk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_gather<<<(unsigned)T, 256, 0, s>>>(static_cast<const uint16_t*>(x), ld_x, H, tk, xc);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const Operand ox{xc, H, T}, oxt{xc, H, H};  // rows of K = H; columns of K = tokens
  const unsigned th = (unsigned)((H + TN - 1) / TN), tt = (unsigned)((T + TN - 1) / TN);
  for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
    const int64_t n = std::min(pl.piece, V - v0);
    const unsigned tv = (unsigned)((n + TM - 1) / TM);
    const uint16_t* wp = static_cast<const uint16_t*>(w) + v0 * ld_w;
    k_logits_grad<<<dim3(tv, tt), 256, 0, s>>>(Operand{wp, ld_w, n}, ox, (int)H, v0, tk, labels, lse, dloss, d, pl.ldd);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (dw != nullptr) {
      const Operand od{d, pl.ldd, n};
      if (dw_dt == 0)
        k_product<false, true, false><<<dim3(tv, th), 256, 0, s>>>(od, oxt, 0, tk.n,
                                                                   static_cast<uint16_t*>(dw) + v0 * ld_dw, ld_dw,
                                                                   accumulate);
      else
        k_product<false, true, false><<<dim3(tv, th), 256, 0, s>>>(od, oxt, 0, tk.n,
                                                                   static_cast<float*>(dw) + v0 * ld_dw, ld_dw,
                                                                   accumulate);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (dx != nullptr) {
      k_product<true, true, true><<<dim3(tt, th), 256, 0, s>>>(Operand{d, pl.ldd, T}, Operand{wp, ld_w, H}, n, tk.n,
                                                               sum, H, v0 > 0 ? 1 : 0);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (dx == nullptr) return hipSuccess;
  k_dx<<<(unsigned)T, 256, 0, s>>>(sum, H, tk, static_cast<uint16_t*>(dx), ld_dx);
  return hipGetLastError();
}

}  // namespace nvfp4
