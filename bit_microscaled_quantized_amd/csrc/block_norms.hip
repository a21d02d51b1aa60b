// The norms after a block and before the next, with the block's gate and residual
// scale between them, and their backward pass (nvfp4_block_norms,
// nvfp4_block_norms_backward), for gfx950.
//
// Bound by HBM.  A group of G lanes takes one row, lane j its 16-byte vectors j,
// j + G, ..., up to VPT of them, which stay in registers over both of the row's sums
// (and, with codes as output, its maximum); rows wider than a workgroup's registers
// are read once per sum and once more.  Sums are FP32 in a fixed order.
#include "act_device.hpp"
#include "blocks_launch.hpp"
#include "row_codes.hpp"

namespace nvfp4 {

namespace {

struct NormsArgs {
  const void* x;
  const void* residual;
  const void* gate;
  const void* post;
  const void* pre;
  void* h;
  void* y;
  int8_t* codes;
  float* scales;
  float* post_rstd;
  float* pre_rstd;
  int64_t ld_x, ld_r, ld_gate, ld_h, ld_y, ld_codes;
  uint32_t rows, cols, padded;  // padded: cols up to a multiple of 16
  int gamma_f32, sigmoid;
  float eps, scale;
};

__device__ __forceinline__ float rstd_of(float sum, uint32_t cols, float eps) {
  return 1.0f / sqrtf(sum / (float)cols + eps);
}

// n elements of a row's N from column c on that lie inside it
template <int N>
__device__ __forceinline__ int inside(uint64_t c, uint32_t cols) {
  return c < cols ? (int)min((uint64_t)N, cols - c) : 0;
}

template <typename T, bool STREAM>
__device__ __forceinline__ u32x4_t load_or_zero(const T* p, int n) {
  return n > 0 ? load_vec<T, STREAM>(p, n) : u32x4_t{0, 0, 0, 0};
}

// f becomes h: residual + scale * (g * ((x * rstd) * gamma)); elements past the row's end stay 0
template <typename T>
__device__ __forceinline__ void sum_vec(const NormsArgs& a, float* f, u32x4_t r, u32x4_t gate, float rstd, uint32_t c,
                                        int n) {
  constexpr int N = VecOf<T>::N;
  float gm[N], fr[N], fg[N];
#pragma unroll
  for (int i = 0; i < N; i++) gm[i] = 0.0f;
  if (n > 0) load_gamma<N>(a.post, a.gamma_f32, c, n, gm);
  VecOf<T>::unpack(r, fr);
#pragma unroll
  for (int i = 0; i < N; i++) f[i] = (f[i] * rstd) * gm[i];
  if (a.gate != nullptr) {
    VecOf<T>::unpack(gate, fg);
#pragma unroll
    for (int i = 0; i < N; i++) f[i] *= a.sigmoid ? sigmoid(fg[i]) : fg[i];
  }
#pragma unroll
  for (int i = 0; i < N; i++) f[i] = __builtin_fmaf(a.scale, f[i], fr[i]);
}

// f becomes y: (h * rstd) * gamma, zeros past the row's end
template <typename T>
__device__ __forceinline__ void norm_vec(const NormsArgs& a, float* f, float rstd, uint32_t c, int n) {
  constexpr int N = VecOf<T>::N;
  float gm[N];
#pragma unroll
  for (int i = 0; i < N; i++) gm[i] = 0.0f;
  if (n > 0) load_gamma<N>(a.pre, a.gamma_f32, c, n, gm);
#pragma unroll
  for (int i = 0; i < N; i++) f[i] = i < n ? (f[i] * rstd) * gm[i] : 0.0f;
}

template <typename T, int VPT, bool CODES, bool STREAM>
__global__ __launch_bounds__(1024) void k_block_norms(NormsArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  const uint32_t row = blockIdx.x * (blockDim.x / G) + threadIdx.x / G, j = threadIdx.x % G;
  const bool live = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  const T* gr = static_cast<const T*>(a.gate) + (int64_t)row * a.ld_gate;
  u32x4_t vx[VPT], vr[VPT], vg[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? inside<N>(c, a.cols) : 0;
    vx[k] = load_or_zero<T, STREAM>(xr + c, n);
    vr[k] = load_or_zero<T, STREAM>(rr + c, a.residual == nullptr ? 0 : n);
    vg[k] = load_or_zero<T, false>(gr + c, a.gate == nullptr ? 0 : n);
  }
  float f[VPT][N], sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    VecOf<T>::unpack(vx[k], f[k]);
#pragma unroll
    for (int i = 0; i < N; i++) sq = __builtin_fmaf(f[k][i], f[k][i], sq);
  }
  const float post = rstd_of(group_sum(sq, G, red), a.cols, a.eps);
  sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? inside<N>(c, a.cols) : 0;
    sum_vec<T>(a, f[k], vr[k], vg[k], post, c, n);
    if (n > 0 && a.h != nullptr)
      store_vec<T, STREAM>(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(f[k]), n);
#pragma unroll
    for (int i = 0; i < N; i++) sq = __builtin_fmaf(f[k][i], f[k][i], sq);
  }
  const float pre = rstd_of(group_sum(sq, G, red), a.cols, a.eps);
  if (live && j == 0) {
    if (a.post_rstd != nullptr) a.post_rstd[row] = post;
    if (a.pre_rstd != nullptr) a.pre_rstd[row] = pre;
  }
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live ? inside<N>(c, a.cols) : 0;
    norm_vec<T>(a, f[k], pre, c, n);
    if constexpr (CODES)
      m = most_of<N>(f[k], m);
    else if (n > 0)
      store_vec<T, STREAM>(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(f[k]), n);
  }
  if constexpr (CODES) {
    const RowCode q(group_max(m, G, reinterpret_cast<uint32_t*>(red)));
    if (!live) return;
    if (j == 0) a.scales[row] = q.scale;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      if (c < a.padded) store_codes<N>(q, f[k], a.codes + (int64_t)row * a.ld_codes, c);
    }
  }
}

// Wider rows: one workgroup a row, whose elements are formed again from x, the residual
// and the gate for each sum; h is written last (it may be the residual).
template <typename T, bool CODES>
__global__ __launch_bounds__(1024) void k_block_norms_wide(NormsArgs a) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  const uint32_t row = blockIdx.x;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  const T* gr = static_cast<const T*>(a.gate) + (int64_t)row * a.ld_gate;
  auto sum_of = [](const float* f) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) s = __builtin_fmaf(f[i], f[i], s);
    return s;
  };
  float sq = 0.0f;
  for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
    float f[N];
    VecOf<T>::unpack(load_vec(xr + c, inside<N>(c, a.cols)), f);
    sq += sum_of(f);
  }
  const float post = rstd_of(group_sum(sq, 1024, red), a.cols, a.eps);
  auto h_of = [&](uint64_t c, int n, float* f) {
    VecOf<T>::unpack(load_or_zero<T, false>(xr + c, n), f);
    sum_vec<T>(a, f, load_or_zero<T, false>(rr + c, a.residual == nullptr ? 0 : n),
               load_or_zero<T, false>(gr + c, a.gate == nullptr ? 0 : n), post, (uint32_t)c, n);
  };
  sq = 0.0f;
  for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
    float f[N];
    h_of(c, inside<N>(c, a.cols), f);
    sq += sum_of(f);
  }
  const float pre = rstd_of(group_sum(sq, 1024, red), a.cols, a.eps);
  if (threadIdx.x == 0) {
    if (a.post_rstd != nullptr) a.post_rstd[row] = post;
    if (a.pre_rstd != nullptr) a.pre_rstd[row] = pre;
  }
  uint32_t m = 0;
  if constexpr (CODES) {
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      float f[N];
      const int n = inside<N>(c, a.cols);
      h_of(c, n, f);
      norm_vec<T>(a, f, pre, (uint32_t)c, n);
      m = most_of<N>(f, m);
    }
    m = group_max(m, 1024, reinterpret_cast<uint32_t*>(red));
  }
  const RowCode q(m);
  if (CODES && threadIdx.x == 0) a.scales[row] = q.scale;
  for (uint64_t c = threadIdx.x * N; c < (CODES ? a.padded : a.cols); c += 1024 * N) {
    float f[N];
    const int n = inside<N>(c, a.cols);
    h_of(c, n, f);
    if (n > 0 && a.h != nullptr) store_vec(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(f), n);
    norm_vec<T>(a, f, pre, (uint32_t)c, n);
    if constexpr (CODES)
      store_codes<N>(q, f, a.codes + (int64_t)row * a.ld_codes, (uint32_t)c);
    else if (n > 0)
      store_vec(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(f), n);
  }
}

// ---- backward

struct NormsBackArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const void* x;
  const void* gate;
  const void* post;
  const void* pre;
  const float* post_rstd;
  const float* pre_rstd;
  void* dx;
  void* dr;
  void* dgate;         // per row; null where the gate is one row for all
  float* pre_part;     // [gridDim.x][cols] sums of dy * n, or null
  float* post_part;    // the same of d * m (without the gate, where it is one row for all), or null
  int64_t ld_dy, ld_dh, ld_h, ld_x, ld_gate, ld_dx, ld_dr, ld_dgate;
  uint32_t rows, cols;
  int gamma_f32, sigmoid, shared;  // shared: one row of gates for all
  float scale;
};

// A lane's vector of a row, in its way through the backward pass.
template <typename T>
struct BackVec {
  static constexpr int N = VecOf<T>::N;
  // t: in, dh; out, dh + rstd * (dy * gamma - n * mean)
  static __device__ __forceinline__ void inner(float* t, const float* dy, const float* h, const float* gamma, float rstd,
                                               float mean) {
#pragma unroll
    for (int i = 0; i < N; i++)
      t[i] = __builtin_fmaf(rstd, __builtin_fmaf(-(h[i] * rstd), mean, dy[i] * gamma[i]), t[i]);
  }
};

// What the second half takes of t: d (the gradient of o), its sum's term and dgate.
//   d = scale * t * g;  dgate = scale * t * (m * gamma) * g'
template <typename T>
__device__ __forceinline__ void gate_vec(const NormsBackArgs& a, const float* t, const float* m, u32x4_t gate,
                                         const float* gamma, float* d, float* term, float* dgate) {
  constexpr int N = VecOf<T>::N;
  float fg[N];
  if (a.gate != nullptr) VecOf<T>::unpack(gate, fg);
#pragma unroll
  for (int i = 0; i < N; i++) {
    d[i] = a.scale * t[i];
    term[i] = d[i] * m[i];
    if (a.gate != nullptr) {
      const float g = a.sigmoid ? sigmoid(fg[i]) : fg[i];
      dgate[i] = (term[i] * gamma[i]) * (a.sigmoid ? g * (1.0f - g) : 1.0f);
      if (!a.shared) term[i] *= g;
      d[i] *= g;
    }
  }
}

template <typename T, int VPT, bool STREAM>
__global__ __launch_bounds__(1024, 4) void k_block_norms_back(NormsBackArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  extern __shared__ float comb[];
  const int groups = blockDim.x / G;
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  float acc_pre[VPT][N], acc_post[VPT][N];
#pragma unroll
  for (int k = 0; k < VPT; k++)
#pragma unroll
    for (int i = 0; i < N; i++) acc_pre[k][i] = acc_post[k][i] = 0.0f;
  for (uint32_t r0 = blockIdx.x * groups; r0 < a.rows; r0 += gridDim.x * groups) {
    const uint32_t row = r0 + grp;
    const bool live = row < a.rows;
    const float pre = live ? a.pre_rstd[row] : 0.0f, post = live ? a.post_rstd[row] : 0.0f;
    u32x4_t vdy[VPT], vh[VPT], vdh[VPT], vx[VPT], vg[VPT];
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? inside<N>(c, a.cols) : 0;
      vdy[k] = load_or_zero<T, STREAM>(static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy + c, n);
      vh[k] = load_or_zero<T, STREAM>(static_cast<const T*>(a.h) + (int64_t)row * a.ld_h + c, n);
      vdh[k] = load_or_zero<T, STREAM>(static_cast<const T*>(a.dh) + (int64_t)row * a.ld_dh + c,
                                       a.dh == nullptr ? 0 : n);
      vx[k] = load_or_zero<T, STREAM>(static_cast<const T*>(a.x) + (int64_t)row * a.ld_x + c, n);
      vg[k] = load_or_zero<T, false>(static_cast<const T*>(a.gate) + (int64_t)row * a.ld_gate + c,
                                     a.gate == nullptr ? 0 : n);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? inside<N>(c, a.cols) : 0;
      if (n <= 0) continue;
      float dy[N], nh[N], gm[N];
      VecOf<T>::unpack(vdy[k], dy);
      VecOf<T>::unpack(vh[k], nh);
      load_gamma<N>(a.pre, a.gamma_f32, c, n, gm);
#pragma unroll
      for (int i = 0; i < N; i++) {
        nh[i] *= pre;
        s = __builtin_fmaf(dy[i] * gm[i], nh[i], s);
        acc_pre[k][i] = __builtin_fmaf(dy[i], nh[i], acc_pre[k][i]);
      }
    }
    const float mean_pre = group_sum(s, G, red) / (float)a.cols;
    float d[VPT][N];
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? inside<N>(c, a.cols) : 0;
      if (n <= 0) continue;
      float dy[N], h[N], gm[N], t[N], m[N], term[N], dg[N];
      VecOf<T>::unpack(vdy[k], dy);
      VecOf<T>::unpack(vh[k], h);
      VecOf<T>::unpack(vdh[k], t);  // zeros without one
      load_gamma<N>(a.pre, a.gamma_f32, c, n, gm);
      BackVec<T>::inner(t, dy, h, gm, pre, mean_pre);
      if (a.dr != nullptr)
        store_vec<T, STREAM>(static_cast<T*>(a.dr) + (int64_t)row * a.ld_dr + c, VecOf<T>::pack(t), n);
      VecOf<T>::unpack(vx[k], m);
      load_gamma<N>(a.post, a.gamma_f32, c, n, gm);
#pragma unroll
      for (int i = 0; i < N; i++) m[i] *= post;
      gate_vec<T>(a, t, m, vg[k], gm, d[k], term, dg);
      if (a.dgate != nullptr)
        store_vec<T, STREAM>(static_cast<T*>(a.dgate) + (int64_t)row * a.ld_dgate + c, VecOf<T>::pack(dg), n);
#pragma unroll
      for (int i = 0; i < N; i++) {
        acc_post[k][i] += term[i];
        d[k][i] *= gm[i];
        s = __builtin_fmaf(d[k][i], m[i], s);
      }
    }
    const float mean_post = group_sum(s, G, red) / (float)a.cols;
    if (a.dx == nullptr) continue;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = live ? inside<N>(c, a.cols) : 0;
      if (n <= 0) continue;
      float m[N];
      VecOf<T>::unpack(vx[k], m);
#pragma unroll
      for (int i = 0; i < N; i++) m[i] = post * __builtin_fmaf(-(m[i] * post), mean_post, d[k][i]);
      store_vec<T, STREAM>(static_cast<T*>(a.dx) + (int64_t)row * a.ld_dx + c, VecOf<T>::pack(m), n);
    }
  }
  // the groups of a workgroup add their sums in LDS, in order
  for (int half = 0; half < 2; half++) {
    float* part = half == 0 ? a.pre_part : a.post_part;
    if (part == nullptr) continue;
    float* out = part + (int64_t)blockIdx.x * a.cols;
    if (groups == 1) {
#pragma unroll
      for (int k = 0; k < VPT; k++) {
        const uint32_t c = (j + k * G) * N;
#pragma unroll
        for (int i = 0; i < N; i++)
          if (c + i < a.cols) out[c + i] = half == 0 ? acc_pre[k][i] : acc_post[k][i];
      }
      continue;
    }
    __syncthreads();  // the first half's sums are read
    for (int q = 0; q < groups; q++) {
      if (grp == q) {
#pragma unroll
        for (int k = 0; k < VPT; k++)
#pragma unroll
          for (int i = 0; i < N; i++) {
            float* p = comb + (j + k * G) * N + i;
            const float v = half == 0 ? acc_pre[k][i] : acc_post[k][i];
            *p = q == 0 ? v : *p + v;
          }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += blockDim.x) out[c] = comb[c];
  }
}

// Wider rows: one workgroup a row at a time, read for each of its two sums and for its
// outputs; the column sums stay in the workgroup's rows of the workspace (each lane adds
// to its own columns).
template <typename T>
__global__ __launch_bounds__(1024) void k_block_norms_back_wide(NormsBackArgs a) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  float* out_pre = a.pre_part == nullptr ? nullptr : a.pre_part + (int64_t)blockIdx.x * a.cols;
  float* out_post = a.post_part == nullptr ? nullptr : a.post_part + (int64_t)blockIdx.x * a.cols;
  for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float pre = a.pre_rstd[row], post = a.post_rstd[row];
    auto at = [&](const void* p, int64_t ld, uint64_t c, float* f) {
      VecOf<T>::unpack(p == nullptr ? u32x4_t{0, 0, 0, 0}
                                    : load_vec(static_cast<const T*>(p) + (int64_t)row * ld + c, inside<N>(c, a.cols)), f);
    };
    float s = 0.0f;
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      float dy[N], h[N], gm[N], q = 0.0f;
      at(a.dy, a.ld_dy, c, dy);
      at(a.h, a.ld_h, c, h);
      load_gamma<N>(a.pre, a.gamma_f32, (uint32_t)c, inside<N>(c, a.cols), gm);
#pragma unroll
      for (int i = 0; i < N; i++) q = __builtin_fmaf(dy[i] * gm[i], h[i] * pre, q);
      s += q;
    }
    const float mean_pre = group_sum(s, 1024, red) / (float)a.cols;
    // t, m, d times gamma, its sum's term and dgate of one vector
    auto form = [&](uint64_t c, float* t, float* m, float* d, float* term, float* dg) {
      const int n = inside<N>(c, a.cols);
      float dy[N], h[N], gm[N];
      at(a.dy, a.ld_dy, c, dy);
      at(a.h, a.ld_h, c, h);
      at(a.dh, a.ld_dh, c, t);
      at(a.x, a.ld_x, c, m);
      load_gamma<N>(a.pre, a.gamma_f32, (uint32_t)c, n, gm);
      BackVec<T>::inner(t, dy, h, gm, pre, mean_pre);
      load_gamma<N>(a.post, a.gamma_f32, (uint32_t)c, n, gm);
#pragma unroll
      for (int i = 0; i < N; i++) m[i] *= post;
      const u32x4_t gate =
          load_or_zero<T, false>(static_cast<const T*>(a.gate) + (int64_t)row * a.ld_gate + c, a.gate == nullptr ? 0 : n);
      gate_vec<T>(a, t, m, gate, gm, d, term, dg);
#pragma unroll
      for (int i = 0; i < N; i++) d[i] *= gm[i];
    };
    s = 0.0f;
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      float t[N], m[N], d[N], term[N], dg[N], q = 0.0f;
      form(c, t, m, d, term, dg);
#pragma unroll
      for (int i = 0; i < N; i++) q = __builtin_fmaf(d[i], m[i], q);
      s += q;
    }
    const float mean_post = group_sum(s, 1024, red) / (float)a.cols;
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      const int n = inside<N>(c, a.cols);
      float t[N], m[N], d[N], term[N], dg[N], dy[N], h[N];
      form(c, t, m, d, term, dg);
      at(a.dy, a.ld_dy, c, dy);
      at(a.h, a.ld_h, c, h);
      const bool first = row == blockIdx.x;
#pragma unroll
      for (int i = 0; i < N; i++) {
        if (i >= n) continue;
        if (out_pre != nullptr) out_pre[c + i] = __builtin_fmaf(dy[i], h[i] * pre, first ? 0.0f : out_pre[c + i]);
        if (out_post != nullptr) out_post[c + i] = term[i] + (first ? 0.0f : out_post[c + i]);
      }
#pragma unroll
      for (int i = 0; i < N; i++) m[i] = post * __builtin_fmaf(-m[i], mean_post, d[i]);
      if (a.dr != nullptr) store_vec(static_cast<T*>(a.dr) + (int64_t)row * a.ld_dr + c, VecOf<T>::pack(t), n);
      if (a.dgate != nullptr)
        store_vec(static_cast<T*>(a.dgate) + (int64_t)row * a.ld_dgate + c, VecOf<T>::pack(dg), n);
      if (a.dx != nullptr) store_vec(static_cast<T*>(a.dx) + (int64_t)row * a.ld_dx + c, VecOf<T>::pack(m), n);
    }
  }
}

// The column sums, in the partial rows' order: 32 slices of rows per column, added in
// LDS.  Half of the grid takes each.  A gate that is one row for all comes in here: S =
// sum_r scale * t * m gives dpost_gamma = g S and dgate = post_gamma S g'.
struct SumArgs {
  const float* pre_part;
  const float* post_part;
  const void* gate;  // where it is one row for all
  const void* post;
  float* dpre;
  float* dpost;
  float* dgate;
  uint32_t parts, cols;
  int dt_f32, gamma_f32, sigmoid;
};
__device__ __forceinline__ float one_of(const void* p, int f32, uint32_t c) {
  return f32 ? static_cast<const float*>(p)[c] : VecOf<uint16_t>::one(static_cast<const uint16_t*>(p) + c);
}
constexpr int SLICES = 32;
__global__ __launch_bounds__(SLICES * 32) void k_column_sums(SumArgs a) {
  __shared__ float part[SLICES][32];
  const uint32_t lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const uint32_t p0 = a.parts * slice / SLICES, p1 = a.parts * (slice + 1) / SLICES;
  const bool post = (blockIdx.x & 1) != 0;
  const float* from = post ? a.post_part : a.pre_part;
  if (from == nullptr) return;
  for (uint64_t base = (blockIdx.x >> 1) * 32; base < a.cols; base += (uint64_t)(gridDim.x >> 1) * 32) {
    const uint64_t c = base + lane;
    float s = 0.0f;
    if (c < a.cols) {
#pragma unroll 8
      for (uint32_t p = p0; p < p1; p++) s += from[(int64_t)p * a.cols + c];
    }
    __syncthreads();  // the last columns' sums are read
    part[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || c >= a.cols) continue;
    s = 0.0f;
#pragma unroll
    for (int q = 0; q < SLICES; q++) s += part[q][lane];
    if (!post) {
      a.dpre[c] = s;
      continue;
    }
    float g = 1.0f, slope = 1.0f;
    if (a.parts == 0) {  // no rows
      if (a.dgate != nullptr) a.dgate[c] = 0.0f;
      if (a.dpost != nullptr) a.dpost[c] = 0.0f;
      continue;
    }
    if (a.gate != nullptr) {
      g = one_of(a.gate, a.dt_f32, (uint32_t)c);
      if (a.sigmoid) {
        g = sigmoid(g);
        slope = g * (1.0f - g);
      }
    }
    if (a.dgate != nullptr) a.dgate[c] = (s * one_of(a.post, a.gamma_f32, (uint32_t)c)) * slope;
    if (a.dpost != nullptr) a.dpost[c] = g * s;
  }
}

constexpr int64_t kCus = 256;

// Shape of a backward pass of vectors of N elements: rows (groups of G lanes) per
// workgroup, and workgroups, each with one row of partial sums for each gain.
struct BackShape {
  RowShape row;
  int groups;
  int64_t parts;
};
BackShape back_shape(int64_t rows, int64_t cols, int N) {
  BackShape b;
  b.row = row_shape((cols + N - 1) / N, 1);
  if (b.row.vpt * N > 16) b.row = RowShape{0, 0};  // beyond the registers
  if (b.row.vpt == 0) return BackShape{b.row, 1, std::min<int64_t>(rows, kCus)};
  b.groups = (int)std::min<int64_t>(std::max(1, 512 / b.row.G), rows);
  b.parts = std::min((rows + b.groups - 1) / b.groups, 2 * kCus);
  return b;
}

template <typename T>
hipError_t norms_back_t(const NormsBackArgs& a, const BackShape& b, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  if (b.row.vpt == 0) {
    k_block_norms_back_wide<T><<<(unsigned)b.parts, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const bool stream = (int64_t)a.rows * a.cols * 6 * (int64_t)sizeof(T) >= kStreamBytes;
  const int lds = b.groups == 1 ? 0 : b.row.G * b.row.vpt * N * (int)sizeof(float);
  with_vpt(b.row.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value * N <= 16 ? vpt.value : 1;  // what back_shape picks
    if (stream)
      k_block_norms_back<T, VPT, true><<<(unsigned)b.parts, b.groups * b.row.G, lds, s>>>(a, b.row.G);
    else
      k_block_norms_back<T, VPT, false><<<(unsigned)b.parts, b.groups * b.row.G, lds, s>>>(a, b.row.G);
  });
  return hipGetLastError();
}

template <typename T, bool CODES>
hipError_t norms_t(const NormsArgs& a, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const int64_t vecs = ((CODES ? (int64_t)a.padded : (int64_t)a.cols) + N - 1) / N;
  const RowShape r = row_shape(vecs, a.rows >= 1024 && vecs > 128 ? 2 : 1);
  if (r.vpt == 0 || r.vpt > 5) {
    k_block_norms_wide<T, CODES><<<a.rows, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const int threads = r.G < 64 ? 256 / r.G * r.G : r.G;
  const unsigned grid = (a.rows + threads / r.G - 1) / (threads / r.G);
  const bool stream = (int64_t)a.rows * a.cols * 4 * (int64_t)sizeof(T) >= kStreamBytes;
  with_vpt(r.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value <= 5 ? vpt.value : 1;
    if (stream)
      k_block_norms<T, VPT, CODES, true><<<grid, threads, 0, s>>>(a, r.G);
    else
      k_block_norms<T, VPT, CODES, false><<<grid, threads, 0, s>>>(a, r.G);
  });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norms(const void* x, const void* residual, const void* gate, int dt, int64_t rows,
                              int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_gate, int gate_act,
                              const void* post_gamma, const void* pre_gamma, int gamma_dt, float eps, float scale,
                              void* h, int64_t ld_h, void* y, int64_t ld_y, int8_t* codes, int64_t ld_codes,
                              float* scales, float* post_rstd, float* pre_rstd, hipStream_t s) {
  const NormsArgs a{x,     residual, gate, post_gamma, pre_gamma, h,        y,     codes,    scales,
                    post_rstd, pre_rstd, ld_x, ld_r,   ld_gate,   ld_h,     ld_y,  ld_codes, (uint32_t)rows,
                    (uint32_t)cols, (uint32_t)((cols + 15) / 16 * 16), gamma_dt, gate_act, eps, scale};
  if (dt == 0) return y == nullptr ? norms_t<uint16_t, true>(a, s) : norms_t<uint16_t, false>(a, s);
  return y == nullptr ? norms_t<float, true>(a, s) : norms_t<float, false>(a, s);
}

int64_t block_norms_back_workspace(int64_t rows, int64_t cols) {
  if (rows == 0) return 0;
  const int64_t parts = std::max(back_shape(rows, cols, 8).parts, back_shape(rows, cols, 4).parts);
  return 2 * parts * cols * (int64_t)sizeof(float);
}

hipError_t launch_block_norms_back(const void* dy, const void* dh, const void* h, const void* x, const void* gate,
                                   int dt, int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_dh, int64_t ld_h,
                                   int64_t ld_x, int64_t ld_gate, int gate_act, const void* post_gamma,
                                   const void* pre_gamma, int gamma_dt, const float* post_rstd, const float* pre_rstd,
                                   float scale, void* dx, int64_t ld_dx, void* dresidual, int64_t ld_dr, void* dgate,
                                   int64_t ld_dgate, float* dpost_gamma, float* dpre_gamma, void* workspace,
                                   hipStream_t s) {
  const bool shared = gate != nullptr && ld_gate == 0;
  float* dgate_sum = shared ? static_cast<float*>(dgate) : nullptr;
  const bool sums = dpre_gamma != nullptr || dpost_gamma != nullptr || dgate_sum != nullptr;
  int64_t parts = 0;
  float* pre_part = nullptr;
  float* post_part = nullptr;
  if (rows > 0) {
    const BackShape b = back_shape(rows, cols, dt == 0 ? 8 : 4);
    parts = b.parts;
    pre_part = dpre_gamma == nullptr ? nullptr : static_cast<float*>(workspace);
    post_part = dpost_gamma == nullptr && dgate_sum == nullptr ? nullptr : static_cast<float*>(workspace) + parts * cols;
    const NormsBackArgs a{dy,        dh,        h,     x,     gate,    post_gamma, pre_gamma,      post_rstd,
                          pre_rstd,  dx,        dresidual, shared ? nullptr : dgate, pre_part, post_part, ld_dy, ld_dh,
                          ld_h,      ld_x,      ld_gate, ld_dx, ld_dr, ld_dgate,   (uint32_t)rows, (uint32_t)cols,
                          gamma_dt,  gate_act,  shared ? 1 : 0, scale};
    const hipError_t e = dt == 0 ? norms_back_t<uint16_t>(a, b, s) : norms_back_t<float>(a, b, s);
    if (e != hipSuccess) return e;
  } else if (sums) {  // no rows: the sums are zero (pointers only say which are asked for)
    pre_part = dpre_gamma;
    post_part = dpost_gamma != nullptr ? dpost_gamma : dgate_sum;
  }
  if (!sums) return hipSuccess;
  const SumArgs a{pre_part,    post_part,   shared ? gate : nullptr, post_gamma, dpre_gamma,
                  dpost_gamma, dgate_sum,   (uint32_t)parts,         (uint32_t)cols, dt,
                  gamma_dt,    gate_act};
  const unsigned grid = 2 * (unsigned)std::min<int64_t>((cols + 31) / 32, 1 << 20);  // lanes of a launch fit 32 bits
  k_column_sums<<<grid, SLICES * 32, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
