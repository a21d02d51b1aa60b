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
// (8 BF16 or 4 FP32 elements), up to VPT of them.  G is 16 or 32, where several
// rows share a wave, or a multiple of 64, chosen per launch to fit the row.  Sums
// are FP32: each lane adds its own elements, lanes are added by a butterfly, waves
// through LDS, always in the same order.
#include "layers_device.hpp"
#include "layers_launch.hpp"
#include "per_device.hpp"
#include "rows_device.hpp"

namespace nvfp4 {

namespace {

constexpr int MXB = 32;  // columns per block of the 8-bit output

// ---- dropout

// Rows are cut into equal segments of up to U vectors a lane.  Narrow rows share a
// workgroup, 1 << lg lanes each (lg < 8); wider ones take a workgroup per segment.
constexpr int DROP_U = 4;

template <typename T, bool STREAM>
__global__ __launch_bounds__(256) void k_dropout(const T* x, int64_t ld_x, T* y, int64_t ld_y, uint32_t rows,
                                                 uint32_t cols, uint32_t segs, uint32_t seg_vecs, int lg, Dropout d) {
  constexpr int N = VecOf<T>::N;
  const uint32_t rb = blockIdx.x / segs, seg = blockIdx.x - rb * segs;
  const uint32_t lanes = lg < 8 ? 1u << lg : blockDim.x;
  const uint32_t row = lg < 8 ? rb * (256u >> lg) + (threadIdx.x >> lg) : rb;
  if (row >= rows) return;
  const uint32_t j = lg < 8 ? threadIdx.x & (lanes - 1) : threadIdx.x;
  const T* xr = x + (int64_t)row * ld_x;
  T* yr = y + (int64_t)row * ld_y;
  u32x4_t v[DROP_U];
  int n[DROP_U];
#pragma unroll
  for (int u = 0; u < DROP_U; u++) {
    const uint32_t at = j + u * lanes;  // vector of the segment
    const int64_t c = ((int64_t)seg * seg_vecs + at) * N;
    n[u] = at < seg_vecs ? (int)min((int64_t)N, (int64_t)cols - c) : 0;
    if (n[u] > 0) v[u] = load_vec<T, STREAM>(xr + c, n[u]);
  }
#pragma unroll
  for (int u = 0; u < DROP_U; u++) {
    if (n[u] <= 0) continue;
    const uint32_t c = (seg * seg_vecs + j + u * lanes) * N;
    float f[N];
    VecOf<T>::unpack(v[u], f);
    drop<N>(f, row * cols + c, d);
    store_vec<T, STREAM>(yr + c, VecOf<T>::pack(f), n[u]);
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
__device__ __forceinline__ void sum_vec(const NormArgs& a, u32x4_t x, u32x4_t r, uint32_t row, uint32_t c, float* h) {
  constexpr int N = VecOf<T>::N;
  VecOf<T>::unpack(x, h);
  if (a.drop.cut != 0) drop<N>(h, row * a.cols + c, a.drop);
  if (a.residual != nullptr) {
    float f[N];
    VecOf<T>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < N; i++) h[i] = f[i] + h[i];
  }
}

// Rows of up to G * VPT vectors, held in registers; all of a row's loads are in
// flight at once.
template <typename T, int VPT, bool MX, bool STREAM>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  const uint32_t row = blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
  const uint32_t j = threadIdx.x % G;
  const bool live = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  u32x4_t vx[VPT], vr[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? (int)a.cols - (int)c : 0;
    vx[k] = vr[k] = u32x4_t{0, 0, 0, 0};
    if (n > 0) {
      vx[k] = load_vec<T, STREAM>(xr + c, n);
      if (a.residual != nullptr) vr[k] = load_vec<T, STREAM>(rr + c, n);
    }
  }
  float h[VPT][N];
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    // elements past the row's end were loaded as zeros and stay zeros
    sum_vec<T>(a, vx[k], vr[k], row, (j + k * G) * N, h[k]);
#pragma unroll
    for (int i = 0; i < N; i++) sq = __builtin_fmaf(h[k][i], h[k][i], sq);
  }
  sq = group_sum(sq, G, red);
  const float rstd = 1.0f / sqrtf(sq / (float)a.cols + a.eps);
  if (live && j == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? (int)a.cols - (int)c : 0;
    if (n > 0 && a.h != nullptr)
      store_vec<T, STREAM>(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(h[k]), n);
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
      if (n > 0) store_vec<T, STREAM>(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(h[k]), n);
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
    sum_vec<T>(a, load_vec(xr + c, n), a.residual == nullptr ? u32x4_t{0, 0, 0, 0} : load_vec(rr + c, n), row,
               (uint32_t)c, h);
#pragma unroll
    for (int i = 0; i < N; i++) s = __builtin_fmaf(h[i], h[i], s);
    sq += s;
  }
  sq = group_sum(sq, 1024, red);
  const float rstd = 1.0f / sqrtf(sq / (float)a.cols + a.eps);
  if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[row] = rstd;
  for (uint64_t base = 0; base < a.cols; base += 1024 * N) {
    const int64_t c = base + threadIdx.x * N;
    const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
    float h[N], g[N];
#pragma unroll
    for (int i = 0; i < N; i++) h[i] = g[i] = 0.0f;
    if (n > 0) {
      sum_vec<T>(a, load_vec(xr + c, n), a.residual == nullptr ? u32x4_t{0, 0, 0, 0} : load_vec(rr + c, n), row,
                 (uint32_t)c, h);
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

// g of one vector: in, dh; out, dh + rstd * (dy * gamma - n * mean), n = h * rstd.
template <int N>
__device__ __forceinline__ void back_vec(float* g, const float* dy, const float* h, const float* gamma, float rstd,
                                         float mean) {
#pragma unroll
  for (int i = 0; i < N; i++)
    g[i] = __builtin_fmaf(rstd, __builtin_fmaf(-(h[i] * rstd), mean, dy[i] * gamma[i]), g[i]);
}

// Stores dresidual and dx of one vector.
template <typename T, bool STREAM>
__device__ __forceinline__ void back_store(const NormBackArgs& a, uint32_t row, uint32_t c, int n, float* g) {
  if (a.dr != nullptr) store_vec<T, STREAM>(static_cast<T*>(a.dr) + (int64_t)row * a.ld_dr + c, VecOf<T>::pack(g), n);
  if (a.dx != nullptr) {
    if (a.drop.cut != 0) drop<VecOf<T>::N>(g, row * a.cols + c, a.drop);
    store_vec<T, STREAM>(static_cast<T*>(a.dx) + (int64_t)row * a.ld_dx + c, VecOf<T>::pack(g), n);
  }
}

// A lane's vectors of a row: dy, h and dh.
template <int VPT>
struct BackRow {
  u32x4_t dy[VPT], h[VPT], dh[VPT];
  float rstd;
};

// Rows of up to G * VPT vectors: each group of G lanes walks rows with a stride,
// its dgamma sums in registers (FP32 rows of five vectors a lane or more, where a
// group is the workgroup, in LDS: the registers hold three tensors' vectors); the
// groups of a workgroup add theirs in LDS (G VPT N floats) in order, and the
// workgroup writes one row of partial sums.
//
// Loads and stores complete in one order, so loads that follow a row's stores
// wait for them as well.  Where the registers hold two rows' vectors (AHEAD), the
// next row's loads are issued a whole row ahead, and gamma, which would queue
// behind them, stays in registers; other rows load dh between the two passes.  Rows
// of one vector a lane run six waves a SIMD: two workgroups of ten waves put six on
// some of them.  MI355X, BF16: 8192 x 5120 82 us (5.1 TB/s; without the load ahead
// 92), 32768 x 2048 114 (139), 4096 x 8192 72 (79); FP32 1023 x 20479, one row a CU
// and nothing ahead, 102 us (4.1 TB/s).
template <typename T, int VPT, bool STREAM, bool WAVES>
__global__ __launch_bounds__(1024, VPT * VecOf<T>::N <= 8 ? 6 : 4) void k_rms_norm_back(NormBackArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  extern __shared__ float comb[];
  const int groups = blockDim.x / G;
  // WAVES: a group is whole waves, so its row is the same all over a wave
  const int at = threadIdx.x / G, grp = WAVES ? __builtin_amdgcn_readfirstlane(at) : at, j = threadIdx.x % G;
  constexpr bool IN_LDS = N == 4 && VPT >= 5;
  constexpr bool AHEAD = VPT * 8 <= 2 * N;
  float acc[IN_LDS ? 1 : VPT][N], gamma[AHEAD ? VPT : 1][N];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < N; i++) gamma[k][i] = 0.0f;
      if (c < a.cols) load_gamma<N>(a.gamma, a.gamma_f32, c, (int)(a.cols - c), gamma[k]);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
      if constexpr (IN_LDS)
        comb[c + i] = 0.0f;
      else
        acc[k][i] = 0.0f;
    }
  }
  auto load = [&](uint32_t r0, BackRow<VPT>& v) {
    const uint32_t row = r0 + grp;
    const bool live = row < a.rows;
    v.rstd = live ? a.rstd[row] : 0.0f;
    const T* dyr = static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy;
    const T* hr = static_cast<const T*>(a.h) + (int64_t)row * a.ld_h;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? (int)a.cols - (int)c : 0;
      v.dy[k] = v.h[k] = u32x4_t{0, 0, 0, 0};
      if (n > 0) {
        v.dy[k] = load_vec<T, STREAM>(dyr + c, n);
        v.h[k] = load_vec<T, STREAM>(hr + c, n);
      }
    }
  };
  auto load_dh = [&](uint32_t r0, BackRow<VPT>& v) {
    const uint32_t row = r0 + grp;
    const T* dhr = static_cast<const T*>(a.dh) + (int64_t)row * a.ld_dh;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = row < a.rows && a.dh != nullptr ? (int)a.cols - (int)c : 0;
      v.dh[k] = u32x4_t{0, 0, 0, 0};
      if (n > 0) v.dh[k] = load_vec<T, STREAM>(dhr + c, n);
    }
  };
  const uint32_t step = gridDim.x * groups;
  BackRow<VPT> next;
  if constexpr (AHEAD) {
    load(blockIdx.x * groups, next);
    load_dh(blockIdx.x * groups, next);
  }
  for (uint32_t r0 = blockIdx.x * groups; r0 < a.rows; r0 += step) {
    const uint32_t row = r0 + grp;
    const int cols = row < a.rows ? (int)a.cols : 0;
    BackRow<VPT> v;
    if constexpr (AHEAD) {
      v = next;
      load(r0 + step, next);
      load_dh(r0 + step, next);
    } else {
      load(r0, v);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      if ((int)c >= cols) continue;
      float dy[N], nh[N], g[N];
      VecOf<T>::unpack(v.dy[k], dy);
      VecOf<T>::unpack(v.h[k], nh);
      if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < N; i++) g[i] = gamma[k][i];
      } else {
        load_gamma<N>(a.gamma, a.gamma_f32, c, cols - (int)c, g);
      }
      float* sums = IN_LDS ? comb + c : acc[IN_LDS ? 0 : k];
#pragma unroll
      for (int i = 0; i < N; i++) {
        nh[i] *= v.rstd;
        s = __builtin_fmaf(dy[i] * g[i], nh[i], s);
        sums[i] = __builtin_fmaf(dy[i], nh[i], sums[i]);
      }
    }
    if constexpr (!AHEAD) load_dh(r0, v);
    const float mean = group_sum(s, G, red) / (float)a.cols;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      if ((int)c >= cols) continue;
      float dy[N], h[N], gm[N], g[N];
      VecOf<T>::unpack(v.dy[k], dy);
      VecOf<T>::unpack(v.h[k], h);
      VecOf<T>::unpack(v.dh[k], g);  // zeros without one
      if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < N; i++) gm[i] = gamma[k][i];
      } else {
        load_gamma<N>(a.gamma, a.gamma_f32, c, cols - (int)c, gm);
      }
      back_vec<N>(g, dy, h, gm, v.rstd, mean);
      back_store<T, STREAM>(a, row, c, cols - (int)c, g);
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (IN_LDS) {
    __syncthreads();
  } else if (groups == 1) {
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const int64_t c = (int64_t)(j + k * G) * N;
#pragma unroll
      for (int i = 0; i < N; i++)
        if (c + i < a.cols) out[c + i] = acc[k][i];
    }
    return;
  } else {
    for (int q = 0; q < groups; q++) {
      if (grp == q) {
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
  }
  for (uint32_t c = threadIdx.x; c < a.cols; c += blockDim.x) out[c] = comb[c];
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
    const float mean = group_sum(s, 1024, red) / (float)a.cols;
    if (a.dx == nullptr && a.dr == nullptr) continue;
    for (int64_t c = (int64_t)threadIdx.x * N; c < a.cols; c += 1024 * N) {
      const int n = (int)min((int64_t)N, (int64_t)a.cols - c);
      float dy[N], h[N], gm[N], g[N];
      VecOf<T>::unpack(load_vec(dyr + c, n), dy);
      VecOf<T>::unpack(load_vec(hr + c, n), h);
      load_gamma<N>(a.gamma, a.gamma_f32, (uint32_t)c, n, gm);
      VecOf<T>::unpack(a.dh == nullptr ? u32x4_t{0, 0, 0, 0}
                                       : load_vec(static_cast<const T*>(a.dh) + (int64_t)row * a.ld_dh + c, n), g);
      back_vec<N>(g, dy, h, gm, rstd, mean);
      back_store<T, true>(a, row, (uint32_t)c, n, g);
    }
  }
}

// dgamma[c] = sum of the partial rows, in their order: 32 slices of rows per
// column, added in LDS.
constexpr int DG = 32;
__global__ __launch_bounds__(DG * 32) void k_dgamma(const float* partial, uint32_t parts, uint32_t cols,
                                                    float* dgamma) {
  __shared__ float part[DG][32];
  const uint32_t lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const uint32_t p0 = parts * slice / DG, p1 = parts * (slice + 1) / DG;
  for (uint64_t base = blockIdx.x * 32; base < cols; base += (uint64_t)gridDim.x * 32) {
    const uint64_t c = base + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
      for (uint32_t p = p0; p < p1; p++) s += partial[(int64_t)p * cols + c];
    }
    __syncthreads();  // the last columns' sums are read
    part[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && c < cols) {
      s = 0.0f;
#pragma unroll
      for (int q = 0; q < DG; q++) s += part[q][lane];
      dgamma[c] = s;
    }
  }
}

// A backward pass keeps about two workgroups of 640 lanes on each CU of a 256-CU
// MI355X, or one of up to 1024 for wider rows: more of them write more partial
// sums than their overlap gains (8192 x 5120, before loads went ahead: 92 us at 512 workgroups, 115 at 1024).
// Six waves a SIMD hold two workgroups of up to 768 lanes; rows that would take more than
// 640 run level with one vector a lane in 768 or two in half as many (two against one: BF16
// 8192 x 5248 84.0 us against 83.5, 8192 x 6144 97.1 / 97.3, 1000 x 6144 24.2 / 22.8;
// FP32 4096 x 3000 53.9 / 50.5, but 1023 x 24576, where the same bound sets how many
// workgroups there are, 194 / 215).
constexpr int64_t kCus = 256;
constexpr int kBackThreads = 640;

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
  const int64_t segs = (vecs + 256 * DROP_U - 1) / (256 * DROP_U);
  const int64_t seg_vecs = (vecs + segs - 1) / segs;
  const int threads = lg < 8 ? 256 : (int)((seg_vecs + 64 * DROP_U - 1) / (64 * DROP_U) * 64);
  const int64_t rpb = lg < 8 ? 256 >> lg : 1;
  const unsigned grid = (unsigned)((rows + rpb - 1) / rpb * segs);
  const T* xp = static_cast<const T*>(x);
  T* yp = static_cast<T*>(y);
  if (rows * cols * 2 * (int64_t)sizeof(T) >= kStreamBytes)
    k_dropout<T, true><<<grid, threads, 0, s>>>(xp, ld_x, yp, ld_y, (uint32_t)rows, (uint32_t)cols, (uint32_t)segs,
                                                (uint32_t)seg_vecs, lg, d);
  else
    k_dropout<T, false><<<grid, threads, 0, s>>>(xp, ld_x, yp, ld_y, (uint32_t)rows, (uint32_t)cols, (uint32_t)segs,
                                                 (uint32_t)seg_vecs, lg, d);
  return hipGetLastError();
}

// Two vectors a lane stream best, one finishes a few rows soonest.
constexpr int64_t kManyRows = 1024;

template <typename T, bool MX>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const int64_t vecs = ((int64_t)a.cols + N - 1) / N;
  const RowShape r = row_shape(vecs, a.rows >= kManyRows && vecs > 128 ? 2 : 1);
  if (r.vpt == 0) {
    k_rms_norm_wide<T, MX><<<a.rows, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const int rows = std::max(1, 256 / r.G);  // of a workgroup, where they are narrow
  const int threads = r.G < 64 ? rows * r.G : r.G;
  const unsigned grid = (a.rows + threads / r.G - 1) / (threads / r.G);
  const bool stream = (int64_t)a.rows * a.cols * 4 * (int64_t)sizeof(T) >= kStreamBytes;
  with_vpt(r.vpt, [&](auto vpt) {
    if (stream)
      k_rms_norm<T, vpt.value, MX, true><<<grid, threads, 0, s>>>(a, r.G);
    else
      k_rms_norm<T, vpt.value, MX, false><<<grid, threads, 0, s>>>(a, r.G);
  });
  return hipGetLastError();
}

// Rows that a group of lanes takes in turn where one workgroup does the whole pass:
// more take longer than a second launch (8 x 2048, two each: 7.5 us against 7.7 in
// two launches; 4 x 5120, four: 10.0 against 8.2).
constexpr int kAloneRows = 2;

// Shape of a backward pass of vectors of N elements: rows (groups of G lanes) per
// workgroup, and workgroups, each with one row of partial sums.
struct BackShape {
  RowShape row;
  int groups;
  int64_t parts;
};
BackShape back_shape(int64_t rows, int64_t cols, int N) {
  BackShape b;
  const int64_t vecs = (cols + N - 1) / N;
  b.row = row_shape(vecs, vecs <= kBackThreads ? 1 : 2);
  // Beyond the registers.  FP32 rows of eight vectors a lane are past the limit already and
  // spill 59 of them (1023 x 20479, five vectors, 103 us; 1023 x 20484, eight, 183; 1023 x
  // 32768 225, and 33000 columns read twice 248).  BF16 8192 x 24576 387 us, 24584 columns
  // read twice 1090.
  if (b.row.vpt * N > 32) b.row = RowShape{0, 0};
  if (b.row.vpt == 0) return BackShape{b.row, 1, std::min<int64_t>(rows, kCus)};
  // a few rows: one workgroup, whose sums are dgamma itself, ends before a second launch would
  const int all = 1024 / b.row.G;
  if (rows <= kAloneRows * all) return BackShape{b.row, (int)std::min<int64_t>(rows, all), 1};
  b.groups = std::max(1, 512 / b.row.G);
  const int64_t most = b.row.G * b.groups <= kBackThreads ? 2 * kCus : kCus;
  // few rows: two or more of them to each partial row
  if (rows <= 2 * kCus && b.row.G <= 512) b.groups = std::max(b.groups, 2);
  b.groups = (int)std::min<int64_t>(b.groups, rows);
  b.parts = std::min((rows + b.groups - 1) / b.groups, most);
  return b;
}

// LDS of a row's sums at most: 1024 lanes of eight FP32 vectors.
constexpr int kMostSums = 128 * 1024;

template <typename T>
hipError_t norm_back_t(const NormBackArgs& a, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const BackShape b = back_shape(a.rows, a.cols, N);
  const RowShape r = b.row;
  const int groups = b.groups;
  const int64_t parts = b.parts;
  if (r.vpt == 0) {
    k_rms_norm_back_wide<T><<<(unsigned)parts, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const bool stream = (int64_t)a.rows * a.cols * 5 * (int64_t)sizeof(T) >= kStreamBytes;
  const int lds = groups == 1 && !(N == 4 && r.vpt >= 5) ? 0 : r.G * r.vpt * N * (int)sizeof(float);
  hipError_t e = hipSuccess;
  with_vpt(r.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value * N <= 32 ? vpt.value : 1;  // what back_shape picks
    auto* kernel = stream ? &k_rms_norm_back<T, VPT, true, true> : &k_rms_norm_back<T, VPT, false, true>;
    if constexpr (VPT == 1)
      if (r.G < 64) kernel = stream ? &k_rms_norm_back<T, 1, true, false> : &k_rms_norm_back<T, 1, false, false>;
    if (lds > 64 * 1024) {
      static std::atomic<uint64_t> done{0};
      e = allow_lds(done, kMostSums, &k_rms_norm_back<T, VPT, true, true>, &k_rms_norm_back<T, VPT, false, true>);
    }
    if (e == hipSuccess) kernel<<<(unsigned)parts, groups * r.G, lds, s>>>(a, r.G);
  });
  return e == hipSuccess ? hipGetLastError() : e;
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

int64_t rms_norm_back_workspace(int64_t rows, int64_t cols) {
  if (rows == 0) return 0;
  const int64_t parts = std::max(back_shape(rows, cols, 8).parts, back_shape(rows, cols, 4).parts);
  return parts * cols * (int64_t)sizeof(float);
}

hipError_t launch_rms_norm_back(const void* dy, const void* dh, const void* h, int dt, int64_t rows, int64_t cols,
                                int64_t ld_dy, int64_t ld_dh, int64_t ld_h, const void* gamma, int gamma_dt,
                                const float* rstd, float p, uint64_t seed, void* dx, int64_t ld_dx, void* dresidual,
                                int64_t ld_dr, float* dgamma, void* workspace, hipStream_t s) {
  const int64_t parts = rows == 0 ? 0 : back_shape(rows, cols, dt == 0 ? 8 : 4).parts;
  float* partial = dgamma == nullptr ? nullptr : parts == 1 ? dgamma : static_cast<float*>(workspace);
  if (rows > 0) {
    NormBackArgs a{dy,   dh,    h,     gamma, rstd,           dx,             dresidual, partial,              ld_dy,
                   ld_dh, ld_h, ld_dx, ld_dr, (uint32_t)rows, (uint32_t)cols, gamma_dt,  make_dropout(p, seed)};
    hipError_t e = dt == 0 ? norm_back_t<uint16_t>(a, s) : norm_back_t<float>(a, s);
    if (e != hipSuccess) return e;
  }
  if (dgamma == nullptr || parts == 1) return hipSuccess;
  const unsigned grid = (unsigned)std::min<int64_t>((cols + 31) / 32, 1 << 20);  // lanes of a launch fit 32 bits
  k_dgamma<<<grid, DG * 32, 0, s>>>(partial, (uint32_t)parts, (uint32_t)cols, dgamma);
  return hipGetLastError();
}

}  // namespace nvfp4
