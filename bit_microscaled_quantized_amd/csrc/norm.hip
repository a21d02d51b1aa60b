// Dropout, the residual addition with RMS norm, and its backward pass
// (nvfp4_dropout, nvfp4_rms_norm, nvfp4_rms_norm_backward), for gfx950.
//
// All three are bound by HBM: each element is read once per input and written
// once per output, and the mask is a few integer operations per pair of
// elements.  A row of a norm stays in registers between the sum of its squares
// and its output, so nothing is read twice; a row wider than a workgroup's
// registers hold is read twice instead.
//
// A group of G lanes takes one row, lane j its 16-byte vectors j, j + G, ...
// (8 BF16 or 4 FP32 elements): narrow rows share a wave or a workgroup, wide
// ones take up to 1024 lanes.  Sums are FP32: each lane adds its own elements,
// lanes are added by a butterfly, waves through LDS, always in the same order.
#include "layers_device.hpp"
#include "layers_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int MXB = 32;  // columns per block of the 8-bit output

// Sum over the G lanes of a group (G <= 64: inside a wave; G > 64: the whole
// workgroup, through red[G / 64]); every lane gets the result.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int m = 1; m < (G < 64 ? G : 64); m <<= 1) v += __shfl_xor(v, m, 64);
  if constexpr (G > 64) {
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < G / 64; w++) v += red[w];
  }
  return v;
}

// ---- dropout

// Rows are cut into segments of G * U vectors; a workgroup of 256 lanes takes
// 256 / G segments of consecutive rows (G lanes each).
constexpr int DROP_U = 4;

template <typename T>
__global__ __launch_bounds__(256) void k_dropout(const T* x, int64_t ld_x, T* y, int64_t ld_y, uint32_t rows,
                                                 uint32_t cols, uint32_t segs, int lg, Dropout d) {
  constexpr int N = VecOf<T>::N;
  const uint32_t G = 1u << lg;
  const uint32_t rb = blockIdx.x / segs, seg = blockIdx.x - rb * segs;
  const uint32_t row = rb * (256u >> lg) + (threadIdx.x >> lg);
  if (row >= rows) return;
  const uint32_t j = threadIdx.x & (G - 1);
  const T* xr = x + (int64_t)row * ld_x;
  T* yr = y + (int64_t)row * ld_y;
  u32x4_t v[DROP_U];
  int n[DROP_U];
#pragma unroll
  for (int u = 0; u < DROP_U; u++) {
    const int64_t c = ((int64_t)seg * DROP_U + u) * G * N + (int64_t)j * N;
    n[u] = (int)min((int64_t)N, (int64_t)cols - c);
    if (n[u] > 0) v[u] = load_vec(xr + c, n[u]);
  }
#pragma unroll
  for (int u = 0; u < DROP_U; u++) {
    if (n[u] <= 0) continue;
    const uint32_t c = (seg * DROP_U + u) * G * N + j * N;
    float f[N];
    VecOf<T>::unpack(v[u], f);
    drop<N>(f, row * cols + c, d);
    store_vec(yr + c, VecOf<T>::pack(f), n[u]);
  }
}

// ---- RMS norm

struct NormArgs {
  const void* x;
  const void* residual;
  const void* gamma;
  void* h;
  void* y;
  uint8_t* codes;
  uint8_t* scales;
  float* rstd;
  int64_t ld_x, ld_r, ld_h, ld_y;
  uint32_t rows, cols;
  int gamma_f32;
  float eps;
  Dropout drop;
};

// N values of gamma at column c (n of them inside the row).
template <int N>
__device__ __forceinline__ void load_gamma(const void* gamma, int f32, uint32_t c, int n, float* g) {
  if (f32) {
    const float* p = static_cast<const float*>(gamma) + c;
#pragma unroll
    for (int i = 0; i < N; i += 4) VecOf<float>::unpack(load_vec(p + i, n - i), g + i);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(gamma) + c;
    if constexpr (N == 8) {
      VecOf<uint16_t>::unpack(load_vec(p, n), g);
    } else {
#pragma unroll
      for (int i = 0; i < N; i++) g[i] = i < n ? VecOf<uint16_t>::one(p + i) : 0.0f;
    }
  }
}

// One vector of the norm in 8 bits: 32 / N adjacent lanes hold a block; every
// lane of the wave takes part (f is zero past the row's end).
template <int N>
__device__ __forceinline__ void store_mx8(const float* f, uint32_t c, int n, uint8_t* codes, uint8_t* scales) {
  // the largest magnitude, on the bits: infinities and NaN order above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; i++) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int s = 1; s < MXB / N; s <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s, 64));
  // amax = a * 2^E, 1 <= a < 2: 448 = 1.75 * 2^8, so the exponent is E - 8 for
  // a <= 1.75 and E - 7 above; below 2^-118 it is clamped to -127, which a
  // subnormal's E = -127 gives as well
  int e = (int)(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, -127);
  const bool finite = m < 0x7F800000u;
  if (n <= 0) return;
  // 2^-e for e in [-127, 120], exact
  const float up = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t w[N / 4];
#pragma unroll
  for (int q = 0; q < N / 4; q++) {
    uint32_t d = 0;
    d = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q] * up, f[4 * q + 1] * up, d, false);
    d = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * q + 2] * up, f[4 * q + 3] * up, d, true);
    w[q] = finite ? d : 0x7F7F7F7Fu;
  }
  if (n >= N) {
    if constexpr (N == 8)
      *reinterpret_cast<u32x2_a1*>(codes + c) = u32x2_t{w[0], w[1]};
    else
      *reinterpret_cast<u32_a1*>(codes + c) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (i < n) codes[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if ((c & (MXB - 1)) == 0) scales[c / MXB] = finite ? (uint8_t)(e + 127) : (uint8_t)255;
}

// h = residual + dropout(x) of one vector
template <typename T>
__device__ __forceinline__ void sum_vec(const NormArgs& a, const T* xr, const T* rr, uint32_t row, uint32_t c, int n,
                                        float* h) {
  constexpr int N = VecOf<T>::N;
  VecOf<T>::unpack(load_vec(xr + c, n), h);
  if (a.drop.cut != 0) drop<N>(h, row * a.cols + c, a.drop);
  if (a.residual != nullptr) {
    float r[N];
    VecOf<T>::unpack(load_vec(rr + c, n), r);
#pragma unroll
    for (int i = 0; i < N; i++) h[i] = r[i] + h[i];
  }
}

// Rows of up to G * VPT vectors, held in registers.
template <typename T, int G, int VPT, bool MX>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_rms_norm(NormArgs a) {
  constexpr int N = VecOf<T>::N;
  constexpr int NT = G < 256 ? 256 : G;
  __shared__ float red[NT / 64];
  const uint32_t row = blockIdx.x * (NT / G) + threadIdx.x / G;
  const uint32_t j = threadIdx.x % G;
  const bool live = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  float h[VPT][N];
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? (int)a.cols - (int)c : 0;
#pragma unroll
    for (int i = 0; i < N; i++) h[k][i] = 0.0f;
    if (n > 0) {
      sum_vec<T>(a, xr, rr, row, c, n, h[k]);
      // elements past the row's end were loaded as zeros and stay zeros
    }
#pragma unroll
    for (int i = 0; i < N; i++) sq += h[k][i] * h[k][i];
  }
  sq = group_sum<G>(sq, red);
  const float rstd = 1.0f / sqrtf(sq / (float)a.cols + a.eps);
  if (live && j == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? (int)a.cols - (int)c : 0;
    if (n > 0 && a.h != nullptr)
      store_vec(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(h[k]), n);
    float g[N];
#pragma unroll
    for (int i = 0; i < N; i++) g[i] = 0.0f;
    if (n > 0) load_gamma<N>(a.gamma, a.gamma_f32, c, n, g);
#pragma unroll
    for (int i = 0; i < N; i++) h[k][i] = (MX && i >= n) ? 0.0f : (h[k][i] * rstd) * g[i];
    if constexpr (MX) {
      const uint32_t blocks = (a.cols + MXB - 1) / MXB;
      store_mx8<N>(h[k], c, n, a.codes + (int64_t)row * a.cols, a.scales + (int64_t)row * blocks);
    } else {
      if (n > 0) store_vec(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(h[k]), n);
    }
  }
}

// Rows wider than that: one workgroup per row, x and residual read twice.
template <typename T, bool MX>
__global__ __launch_bounds__(1024) void k_rms_norm_wide(NormArgs a) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  const uint32_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  float sq = 0.0f;
  for (uint64_t base = 0; base < a.cols; base += 1024 * N) {
    const int64_t c = base + threadIdx.x * N;
    const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
    if (n <= 0) continue;
    float h[N], s = 0.0f;
    sum_vec<T>(a, xr, rr, row, (uint32_t)c, n, h);
#pragma unroll
    for (int i = 0; i < N; i++) s += h[i] * h[i];
    sq += s;
  }
  sq = group_sum<1024>(sq, red);
  const float rstd = 1.0f / sqrtf(sq / (float)a.cols + a.eps);
  if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
  for (uint64_t base = 0; base < a.cols; base += 1024 * N) {
    const int64_t c = base + threadIdx.x * N;
    const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
    float h[N], g[N];
#pragma unroll
    for (int i = 0; i < N; i++) h[i] = g[i] = 0.0f;
    if (n > 0) {
      sum_vec<T>(a, xr, rr, row, (uint32_t)c, n, h);
      load_gamma<N>(a.gamma, a.gamma_f32, (uint32_t)c, n, g);
      if (a.h != nullptr) store_vec(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(h), n);
    }
#pragma unroll
    for (int i = 0; i < N; i++) h[i] = (MX && i >= n) ? 0.0f : (h[i] * rstd) * g[i];
    if constexpr (MX) {
      const uint32_t blocks = (a.cols + MXB - 1) / MXB;
      store_mx8<N>(h, (uint32_t)c, n, a.codes + (int64_t)row * a.cols, a.scales + (int64_t)row * blocks);
    } else {
      if (n > 0) store_vec(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(h), n);
    }
  }
}

// ---- backward of the RMS norm

struct NormBackArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const void* gamma;
  const float* rstd;
  void* dx;
  void* dr;
  float* partial;  // [gridDim.x][cols] sums of dgamma, or null
  int64_t ld_dy, ld_dh, ld_h, ld_dx, ld_dr;
  uint32_t rows, cols;
  int gamma_f32;
  Dropout drop;
};

// g of one vector, from gy = dy * gamma, n = h * rstd and the row's mean c of
// gy * n; stores dresidual and dx.
template <typename T>
__device__ __forceinline__ void back_vec(const NormBackArgs& a, uint32_t row, uint32_t c, int n, const float* gy,
                                         const float* nh, float rstd, float mean) {
  constexpr int N = VecOf<T>::N;
  float g[N];
#pragma unroll
  for (int i = 0; i < N; i++) g[i] = rstd * (gy[i] - nh[i] * mean);
  if (a.dh != nullptr) {
    float d[N];
    VecOf<T>::unpack(load_vec(static_cast<const T*>(a.dh) + (int64_t)row * a.ld_dh + c, n), d);
#pragma unroll
    for (int i = 0; i < N; i++) g[i] = d[i] + g[i];
  }
  if (a.dr != nullptr) store_vec(static_cast<T*>(a.dr) + (int64_t)row * a.ld_dr + c, VecOf<T>::pack(g), n);
  if (a.dx != nullptr) {
    if (a.drop.cut != 0) drop<N>(g, row * a.cols + c, a.drop);
    store_vec(static_cast<T*>(a.dx) + (int64_t)row * a.ld_dx + c, VecOf<T>::pack(g), n);
  }
}

// Rows of up to G * VPT vectors: each group of G lanes walks rows with a
// stride, its dgamma sums in registers; the groups of a workgroup add theirs in
// LDS in order, and the workgroup writes one row of partial sums.
template <typename T, int G, int VPT>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_rms_norm_back(NormBackArgs a) {
  constexpr int N = VecOf<T>::N;
  constexpr int NT = G < 256 ? 256 : G;
  constexpr int GROUPS = NT / G;
  __shared__ float red[NT / 64];
  __shared__ float comb[GROUPS > 1 ? G * VPT * N : 1];
  const uint32_t grp = threadIdx.x / G, j = threadIdx.x % G;
  float acc[VPT][N];
#pragma unroll
  for (int k = 0; k < VPT; k++)
#pragma unroll
    for (int i = 0; i < N; i++) acc[k][i] = 0.0f;
  for (uint32_t r0 = blockIdx.x * GROUPS; r0 < a.rows; r0 += gridDim.x * GROUPS) {
    const uint32_t row = r0 + grp;
    const bool live = row < a.rows;
    const float rstd = live ? a.rstd[row] : 0.0f;
    const T* dyr = static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy;
    const T* hr = static_cast<const T*>(a.h) + (int64_t)row * a.ld_h;
    u32x4_t vy[VPT], vh[VPT];
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? (int)a.cols - (int)c : 0;
      vy[k] = vh[k] = u32x4_t{0, 0, 0, 0};
      if (n > 0) {
        vy[k] = load_vec(dyr + c, n);
        vh[k] = load_vec(hr + c, n);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? (int)a.cols - (int)c : 0;
      float dy[N], nh[N], g[N];
      VecOf<T>::unpack(vy[k], dy);
      VecOf<T>::unpack(vh[k], nh);
      if (n > 0) {
        load_gamma<N>(a.gamma, a.gamma_f32, c, n, g);
#pragma unroll
        for (int i = 0; i < N; i++) {
          nh[i] *= rstd;
          s += (dy[i] * g[i]) * nh[i];
          acc[k][i] += dy[i] * nh[i];
        }
      }
    }
    const float mean = group_sum<G>(s, red) / (float)a.cols;
    if (a.dx == nullptr && a.dr == nullptr) continue;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? (int)a.cols - (int)c : 0;
      if (n <= 0) continue;
      float gy[N], nh[N], g[N];
      VecOf<T>::unpack(vy[k], gy);
      VecOf<T>::unpack(vh[k], nh);
      load_gamma<N>(a.gamma, a.gamma_f32, c, n, g);
#pragma unroll
      for (int i = 0; i < N; i++) {
        gy[i] *= g[i];
        nh[i] *= rstd;
      }
      back_vec<T>(a, row, c, n, gy, nh, rstd, mean);
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (GROUPS > 1) {
#pragma unroll 1
    for (int q = 0; q < GROUPS; q++) {
      if ((int)grp == q) {
#pragma unroll
        for (int k = 0; k < VPT; k++)
#pragma unroll
          for (int i = 0; i < N; i++) {
            float* p = comb + (j + k * G) * N + i;
            *p = q == 0 ? acc[k][i] : *p + acc[k][i];
          }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += NT) out[c] = comb[c];
  } else {
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const int64_t c = (int64_t)(j + k * G) * N;
#pragma unroll
      for (int i = 0; i < N; i++)
        if (c + i < a.cols) out[c + i] = acc[k][i];
    }
  }
}

// Wider rows: dy and h are read twice, and the workgroup's dgamma sums stay in
// its own row of the workspace (each lane adds to its own columns).
template <typename T>
__global__ __launch_bounds__(1024) void k_rms_norm_back_wide(NormBackArgs a) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  float* out = a.partial == nullptr ? nullptr : a.partial + (int64_t)blockIdx.x * a.cols;
  for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float rstd = a.rstd[row];
    const T* dyr = static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy;
    const T* hr = static_cast<const T*>(a.h) + (int64_t)row * a.ld_h;
    float s = 0.0f;
    for (int64_t c = (int64_t)threadIdx.x * N; c < a.cols; c += 1024 * N) {
      const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
      float dy[N], nh[N], g[N], t = 0.0f;
      VecOf<T>::unpack(load_vec(dyr + c, n), dy);
      VecOf<T>::unpack(load_vec(hr + c, n), nh);
      load_gamma<N>(a.gamma, a.gamma_f32, (uint32_t)c, n, g);
#pragma unroll
      for (int i = 0; i < N; i++) {
        nh[i] *= rstd;
        t += (dy[i] * g[i]) * nh[i];
        if (out != nullptr && i < n) out[c + i] = row == blockIdx.x ? dy[i] * nh[i] : out[c + i] + dy[i] * nh[i];
      }
      s += t;
    }
    const float mean = group_sum<1024>(s, red) / (float)a.cols;
    if (a.dx == nullptr && a.dr == nullptr) continue;
    for (int64_t c = (int64_t)threadIdx.x * N; c < a.cols; c += 1024 * N) {
      const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
      float gy[N], nh[N], g[N];
      VecOf<T>::unpack(load_vec(dyr + c, n), gy);
      VecOf<T>::unpack(load_vec(hr + c, n), nh);
      load_gamma<N>(a.gamma, a.gamma_f32, (uint32_t)c, n, g);
#pragma unroll
      for (int i = 0; i < N; i++) {
        gy[i] *= g[i];
        nh[i] *= rstd;
      }
      back_vec<T>(a, row, (uint32_t)c, n, gy, nh, rstd, mean);
    }
  }
}

// dgamma[c] = sum of the partial rows, in their order: eight slices of rows per
// column, added in LDS.
__global__ __launch_bounds__(256) void k_dgamma(const float* partial, uint32_t parts, uint32_t cols, float* dgamma) {
  __shared__ float part[8][32];
  const uint32_t lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const uint32_t c = blockIdx.x * 32 + lane;
  const uint32_t p0 = parts * slice / 8, p1 = parts * (slice + 1) / 8;
  float s = 0.0f;
  if (c < cols)
    for (uint32_t p = p0; p < p1; p++) s += partial[(int64_t)p * cols + c];
  part[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; q++) s += part[q][lane];
    dgamma[c] = s;
  }
}

// Workgroups of a backward pass, each with one row of partial sums.
constexpr int64_t kBackGroups = 512;

// f(G, VPT) for rows of `vecs` vectors: the fewest lanes that hold a row with
// at most four vectors each, up to 1024 lanes with eight.  Returns false for a
// wider row.
template <typename F>
bool by_width(int64_t vecs, F&& f) {
  using std::integral_constant;
#define NVFP4_WIDTH(G, VPT)                                                \
  if (vecs <= (G) * (VPT)) {                                               \
    f(integral_constant<int, G>{}, integral_constant<int, VPT>{});         \
    return true;                                                           \
  }
  NVFP4_WIDTH(16, 1)
  NVFP4_WIDTH(32, 1)
  NVFP4_WIDTH(64, 1)
  NVFP4_WIDTH(64, 2)
  NVFP4_WIDTH(256, 1)
  NVFP4_WIDTH(256, 2)
  NVFP4_WIDTH(256, 3)
  NVFP4_WIDTH(512, 2)
  NVFP4_WIDTH(512, 3)
  NVFP4_WIDTH(512, 4)
  NVFP4_WIDTH(1024, 3)
  NVFP4_WIDTH(1024, 4)
  NVFP4_WIDTH(1024, 5)
  NVFP4_WIDTH(1024, 8)
#undef NVFP4_WIDTH
  return false;
}

template <typename T>
hipError_t dropout_t(const void* x, int64_t rows, int64_t cols, int64_t ld_x, void* y, int64_t ld_y, const Dropout& d,
                     hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  if (ld_x == cols && ld_y == cols) {  // one long row: every vector aligned
    cols *= rows;
    rows = 1;
    ld_x = ld_y = cols;
  }
  const int64_t vecs = (cols + N - 1) / N;
  int lg = 4;
  while (lg < 8 && (int64_t(1) << lg) < vecs) lg++;
  const int64_t segs = (vecs + (DROP_U << lg) - 1) / (DROP_U << lg);
  const int64_t rpb = 256 >> lg;
  const int64_t grid = (rows + rpb - 1) / rpb * segs;
  k_dropout<T><<<(unsigned)grid, 256, 0, s>>>(static_cast<const T*>(x), ld_x, static_cast<T*>(y), ld_y,
                                              (uint32_t)rows, (uint32_t)cols, (uint32_t)segs, lg, d);
  return hipGetLastError();
}

template <typename T, bool MX>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const int64_t vecs = ((int64_t)a.cols + N - 1) / N;
  const bool held = by_width(vecs, [&](auto G, auto VPT) {
    constexpr int g = G.value, v = VPT.value, nt = g < 256 ? 256 : g;
    const uint32_t rpb = nt / g;
    k_rms_norm<T, g, v, MX><<<(a.rows + rpb - 1) / rpb, nt, 0, s>>>(a);
  });
  if (!held) k_rms_norm_wide<T, MX><<<a.rows, 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_back_t(const NormBackArgs& a, int64_t parts, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const int64_t vecs = ((int64_t)a.cols + N - 1) / N;
  const bool held = by_width(vecs, [&](auto G, auto VPT) {
    constexpr int g = G.value, v = VPT.value, nt = g < 256 ? 256 : g;
    k_rms_norm_back<T, g, v><<<(unsigned)parts, nt, 0, s>>>(a);
  });
  if (!held) k_rms_norm_back_wide<T><<<(unsigned)parts, 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int dt, int64_t rows, int64_t cols, int64_t ld_x, float p, uint64_t seed,
                          void* y, int64_t ld_y, hipStream_t s) {
  const Dropout d = make_dropout(p, seed);
  return dt == 0 ? dropout_t<uint16_t>(x, rows, cols, ld_x, y, ld_y, d, s)
                 : dropout_t<float>(x, rows, cols, ld_x, y, ld_y, d, s);
}

hipError_t launch_rms_norm(const void* x, const void* residual, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                           int64_t ld_r, const void* gamma, int gamma_dt, float eps, float p, uint64_t seed, void* h,
                           int64_t ld_h, void* y, int64_t ld_y, uint8_t* codes, uint8_t* scales, float* rstd,
                           hipStream_t s) {
  NormArgs a{x,    residual, gamma, h,    y,    codes,          scales,         rstd,          ld_x,
             ld_r, ld_h,     ld_y,  (uint32_t)rows, (uint32_t)cols, gamma_dt, eps, make_dropout(p, seed)};
  if (dt == 0) return y == nullptr ? norm_t<uint16_t, true>(a, s) : norm_t<uint16_t, false>(a, s);
  return y == nullptr ? norm_t<float, true>(a, s) : norm_t<float, false>(a, s);
}

// A workgroup's partial row is worth its write where it sums several rows.
static int64_t back_parts(int64_t rows) { return std::min(rows, kBackGroups); }

int64_t rms_norm_back_workspace(int64_t rows, int64_t cols) { return back_parts(rows) * cols * (int64_t)sizeof(float); }

hipError_t launch_rms_norm_back(const void* dy, const void* dh, const void* h, int dt, int64_t rows, int64_t cols,
                                int64_t ld_dy, int64_t ld_dh, int64_t ld_h, const void* gamma, int gamma_dt,
                                const float* rstd, float p, uint64_t seed, void* dx, int64_t ld_dx, void* dresidual,
                                int64_t ld_dr, float* dgamma, void* workspace, hipStream_t s) {
  const int64_t parts = back_parts(rows);
  float* partial = dgamma == nullptr ? nullptr : static_cast<float*>(workspace);
  if (rows > 0) {
    NormBackArgs a{dy,   dh,    h,     gamma, rstd,           dx,             dresidual, partial,              ld_dy,
                   ld_dh, ld_h, ld_dx, ld_dr, (uint32_t)rows, (uint32_t)cols, gamma_dt,  make_dropout(p, seed)};
    hipError_t e = dt == 0 ? norm_back_t<uint16_t>(a, parts, s) : norm_back_t<float>(a, parts, s);
    if (e != hipSuccess) return e;
  }
  if (dgamma == nullptr) return hipSuccess;
  k_dgamma<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(partial, (uint32_t)parts, (uint32_t)cols, dgamma);
  return hipGetLastError();
}

}  // namespace nvfp4
