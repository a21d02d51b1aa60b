// The norms after a block and before the next, with the block's gate and residual
// scale between them, and their backward pass (nvfp4_block_norms,
// nvfp4_block_norms_backward), for gfx950.
//
// Bound by HBM.  A group of G lanes takes one row, lane j its 16-byte vectors j,
// j + G, ..., up to VPT of them, which stay in registers over both of the row's sums
// (and, with codes as output, its maximum); rows wider than a workgroup's registers
// are read once per sum and once more.  Sums are FP32 in a fixed order.
// 8192 x 5120 BF16 with a gate per row: 420 MB in 68 to 69 us (6.1 TB/s; a copy of tensors of that
// size reaches 6.2), backward 671 MB in 123 to 124 us (5.4 TB/s; 120 and 5.6 without the second
// launch, which adds the sums over rows).
#include "act_device.hpp"
#include "blocks_launch.hpp"
#include "per_device.hpp"
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

// A place in a row, `off` bytes from its start (rows in registers are narrower than 2^17
// columns): where the row is the same all over a wave, a lane then needs no 64-bit
// address for each tensor.
template <typename T, typename P>
__device__ __forceinline__ T* at_row(P* p, uint32_t row, int64_t ld, uint32_t off) {
  T* start = static_cast<T*>(p) + (int64_t)row * ld;
  if constexpr (std::is_const_v<T>)
    return reinterpret_cast<T*>(reinterpret_cast<const uint8_t*>(start) + off);
  else
    return reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(start) + off);
}

// N gains from column c on, n (more than 0) of them inside the row; zeros behind them.
template <int N, bool WHOLE, typename I>
__device__ __forceinline__ void load_gains(const void* gamma, int f32, I c, int n, uint32_t cols, float* g) {
  if constexpr (WHOLE) {
    load_gamma<N>(gamma, f32, (uint32_t)c, N, g);
  } else if (f32) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      VecOf<float>::unpack(load_or_zero<float, false>(static_cast<const float*>(gamma), c + i, n - i, cols), g + i);
  } else if constexpr (N == 8) {
    VecOf<uint16_t>::unpack(load_or_zero<uint16_t, false>(static_cast<const uint16_t*>(gamma), c, n, cols), g);
  } else {
    load_gamma<N>(gamma, 0, (uint32_t)c, n, g);
  }
}

// f becomes h: residual + scale * (g * ((x * rstd) * gamma)); elements past the row's end stay 0
template <typename T, bool WHOLE = false>
__device__ __forceinline__ void sum_vec(const NormsArgs& a, float* f, u32x4_t r, u32x4_t gate, float rstd, uint32_t c,
                                        int n) {
  constexpr int N = VecOf<T>::N;
  float gm[N], fr[N], fg[N];
#pragma unroll
  for (int i = 0; i < N; i++) gm[i] = 0.0f;
  if (n > 0) load_gains<N, WHOLE>(a.post, a.gamma_f32, c, n, a.cols, gm);
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
template <typename T, bool WHOLE = false>
__device__ __forceinline__ void norm_vec(const NormsArgs& a, float* f, float rstd, uint32_t c, int n) {
  constexpr int N = VecOf<T>::N;
  float gm[N];
#pragma unroll
  for (int i = 0; i < N; i++) gm[i] = 0.0f;
  if (n > 0) load_gains<N, WHOLE>(a.pre, a.gamma_f32, c, n, a.cols, gm);
#pragma unroll
  for (int i = 0; i < N; i++) f[i] = i < n ? (f[i] * rstd) * gm[i] : 0.0f;
}

// WHOLE: rows are whole vectors (32768 x 1024 BF16 57 us, 61 with what an end inside one
// takes).
template <typename T, int VPT, bool CODES, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(1024) void k_block_norms(NormsArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ float red[16];
  const uint32_t row = blockIdx.x * (blockDim.x / G) + threadIdx.x / G, j = threadIdx.x % G;
  const bool live = row < a.rows;
  const T* xr = static_cast<const T*>(a.x) + (int64_t)row * a.ld_x;
  const T* rr = static_cast<const T*>(a.residual) + (int64_t)row * a.ld_r;
  const T* gr = static_cast<const T*>(a.gate) + (int64_t)row * a.ld_gate;
  // a vector's elements inside the row, from column c on
  auto part = [&](uint32_t c) { return !live ? 0 : WHOLE ? (c < a.cols ? N : 0) : inside<N>(c, a.cols); };
  u32x4_t vx[VPT], vr[VPT], vg[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = part(c);
    vx[k] = load_row<T, STREAM, WHOLE>(xr, c, n, a.cols);
    vr[k] = load_row<T, STREAM, WHOLE>(rr, c, a.residual == nullptr ? 0 : n, a.cols);
    vg[k] = load_row<T, false, WHOLE>(gr, c, a.gate == nullptr ? 0 : n, a.cols);
  }
  float f[VPT][N], sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    if constexpr (!WHOLE) {
      const int n = part((j + k * G) * N);
      end_row<T>(vx[k], n, a.cols);
      end_row<T>(vr[k], n, a.cols);
      end_row<T>(vg[k], n, a.cols);
    }
    VecOf<T>::unpack(vx[k], f[k]);
#pragma unroll
    for (int i = 0; i < N; i++) sq = __builtin_fmaf(f[k][i], f[k][i], sq);
  }
  const float post = rstd_of(group_sum(sq, G, red), a.cols, a.eps);
  sq = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = part(c);
    sum_vec<T, WHOLE>(a, f[k], vr[k], vg[k], post, c, n);
    if (n > 0 && a.h != nullptr)
      store_vec<T, STREAM>(static_cast<T*>(a.h) + (int64_t)row * a.ld_h + c, VecOf<T>::pack(f[k]), WHOLE ? N : n);
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
    const int n = part(c);
    norm_vec<T, WHOLE>(a, f[k], pre, c, n);
    if constexpr (CODES)
      m = most_of<N>(f[k], m);
    else if (n > 0)
      store_vec<T, STREAM>(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(f[k]), WHOLE ? N : n);
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
    VecOf<T>::unpack(load_or_zero<T, false>(xr, c, inside<N>(c, a.cols), a.cols), f);
    sq += sum_of(f);
  }
  const float post = rstd_of(group_sum(sq, 1024, red), a.cols, a.eps);
  auto h_of = [&](uint64_t c, int n, float* f) {
    VecOf<T>::unpack(load_or_zero<T, false>(xr, c, n, a.cols), f);
    sum_vec<T>(a, f, load_or_zero<T, false>(rr, c, a.residual == nullptr ? 0 : n, a.cols),
               load_or_zero<T, false>(gr, c, a.gate == nullptr ? 0 : n, a.cols), post, (uint32_t)c, n);
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

// Element c of a vector of BF16 or FP32.
__device__ __forceinline__ float one_of(const void* p, int f32, uint32_t c) {
  return f32 ? static_cast<const float*>(p)[c] : VecOf<uint16_t>::one(static_cast<const uint16_t*>(p) + c);
}

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
  void* dgate;  // per row; null where the gate is one row for all
  float* pre_part;     // [gridDim.x][cols] sums of dy * n, or null
  float* post_part;    // the same of d * m (without the gate, where it is one row for all), or null
  int64_t ld_dy, ld_dh, ld_h, ld_x, ld_gate, ld_dx, ld_dr, ld_dgate;
  uint32_t rows, cols;
  int gamma_f32, sigmoid;
  float scale;
};

// t: in, dh; out, dh + rstd * (dy * gamma - n * mean), n = h * rstd
template <int N>
__device__ __forceinline__ void back_vec(float* t, const float* dy, const float* h, const float* gamma, float rstd,
                                         float mean) {
  const float f = -(rstd * mean);
#pragma unroll
  for (int i = 0; i < N; i++) t[i] = __builtin_fmaf(rstd, __builtin_fmaf(h[i], f, dy[i] * gamma[i]), t[i]);
}

// A gate: none, one row for all rows, or one for each, itself or its logistic function.
enum GateKind { kNoGate, kChannel, kToken, kTokenSigmoid };

// What the second half takes of t, for N elements: b = d * gamma, d its gradient of o,
// dgate, and d * m added to sum (without the gate of a channel).  gate: the factor of a
// channel, a token's tensor otherwise.
//   d = scale * t * g;  dgate = scale * t * (m * gamma) * g'
template <int KIND, int N>
__device__ __forceinline__ void gate_vec(float scale, const float* t, const float* m, const float* gate,
                                         const float* gamma, float* b, float* sum, float* dgate) {
#pragma unroll
  for (int i = 0; i < N; i++) {
    const float d = scale * t[i];
    if constexpr (KIND == kToken || KIND == kTokenSigmoid) {
      const float g = KIND == kTokenSigmoid ? sigmoid(gate[i]) : gate[i];
      const float term = d * m[i];
      dgate[i] = term * gamma[i];
      if constexpr (KIND == kTokenSigmoid) dgate[i] *= __builtin_fmaf(-g, g, g);
      sum[i] = __builtin_fmaf(term, g, sum[i]);
      b[i] = (d * g) * gamma[i];
    } else {
      sum[i] = __builtin_fmaf(d, m[i], sum[i]);
      b[i] = (KIND == kChannel ? d * gate[i] : d) * gamma[i];
    }
  }
}

// group_sum with a place in LDS of its own, which every wave has left before the
// workgroup's last barrier but one: one barrier a sum.
__device__ __forceinline__ float group_sum_once(float v, int G, float* red) {
  v = span_sum(v, G);
  if (G > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = G / 64, first = (int)threadIdx.x / G * waves, w = threadIdx.x & 15;
    v = span_sum(w >= first && w < first + waves ? red[w] : 0.0f, 16);
  }
  return v;
}

// A lane's vectors of a row.
template <int VPT>
struct NormsRow {
  u32x4_t dy[VPT], h[VPT], dh[VPT], x[VPT], gate[VPT];
  float pre, post;
};

// Four values of a vector in LDS
__device__ __forceinline__ void lds_four(const float* p, float* f) {
  VecOf<float>::unpack(*reinterpret_cast<const u32x4_t*>(p), f);
}
// Elements 4 u .. 4 u + 3 of a vector, and their place in one
template <typename T>
__device__ __forceinline__ void unpack_four(const u32x4_t& v, int u, float* f) {
  if constexpr (sizeof(T) == 4) {
    VecOf<float>::unpack(v, f);
  } else {
    f[0] = bf16lo(v[2 * u]), f[1] = bf16hi(v[2 * u]), f[2] = bf16lo(v[2 * u + 1]), f[3] = bf16hi(v[2 * u + 1]);
  }
}
template <typename T>
__device__ __forceinline__ void pack_four(u32x4_t& v, int u, const float* f) {
  if constexpr (sizeof(T) == 4) {
    v = VecOf<float>::pack(f);
  } else {
    v[2 * u] = bf16_pack(f[0], f[1]);
    v[2 * u + 1] = bf16_pack(f[2], f[3]);
  }
}

// Another offset for all that the compiler knows: sums of it with the bases of the
// tensors are not kept over the rows.
__device__ __forceinline__ void opaque(uint32_t& off) { asm volatile("" : "+v"(off)); }

// What a vector holds is unknown from here on: the compiler unpacks it again where it is
// used again, rather than keep its elements (twice the registers) over a sum.
__device__ __forceinline__ void packed(u32x4_t& v) { asm volatile("" : "+v"(v)); }
// These sums are needed here: the compiler does not put their additions off to the end
// of the row (and keep both factors until then).
template <int N>
__device__ __forceinline__ void added(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i++) asm volatile("" : "+v"(v[i]));
}

// Rows of up to G * VPT vectors: each group of G lanes walks rows with a stride, its
// column sums in registers; the groups of a workgroup add theirs in LDS in order.
//
// Loads and stores complete in one order, so loads that follow a row's stores wait for
// them as well.  So the gains (and a gate that is one row for all) lie in LDS, in FP32,
// and where the registers hold two rows' vectors (AHEAD) the next row's loads are in
// flight while a row is summed.
//
// WAVES: a group is whole waves, so its row is the same all over a wave.
template <typename T, int VPT, int KIND, bool STREAM, bool WAVES>
__global__ __launch_bounds__(1024, 4) void k_block_norms_back(NormsBackArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  constexpr bool AHEAD = VPT * N <= 8, TOKEN = KIND == kToken || KIND == kTokenSigmoid;
  __shared__ float red[2][16];
  extern __shared__ __align__(16) float gains[];
  const int groups = blockDim.x / G;
  const int at = threadIdx.x / G, grp = WAVES ? __builtin_amdgcn_readfirstlane(at) : at, j = threadIdx.x % G;
  const uint32_t width = (uint32_t)(G * VPT) * N;  // columns of the vectors in LDS, zeros past cols
  float acc_pre[VPT][N], acc_post[VPT][N];
  // A row's last vector may end past it: it is read as the last whole one and shifted (so
  // are the vectors behind it, by a whole one).
  uint32_t from[VPT], to[VPT];  // bytes
  int sh[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
#pragma unroll
    for (int i = 0; i < N; i++) acc_pre[k][i] = acc_post[k][i] = 0.0f;
    const uint32_t c = (j + k * G) * N;
    from[k] = min(c, a.cols - N);
    sh[k] = (int)min(c - from[k], (uint32_t)N);
    from[k] *= (uint32_t)sizeof(T);
    to[k] = c * (uint32_t)sizeof(T);
  }
  // without a dh, dy is read in its place and cleared
  const void* dh = a.dh == nullptr ? a.dy : a.dh;
  const int64_t ld_dh = a.dh == nullptr ? a.ld_dy : a.ld_dh;
  const uint32_t dh_mask = a.dh == nullptr ? 0u : ~0u;
  // Rows past the last are read from it (whatever follows, as many loads are in flight, which
  // is what the waits for the row before them count) and cleared below.
  auto load = [&](uint32_t r0, NormsRow<VPT>& v) {
    const uint32_t row = min(r0 + grp, a.rows - 1);
    v.pre = a.pre_rstd[row];
    v.post = a.post_rstd[row];
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      opaque(from[k]);
      v.dy[k] = load_vec<T, STREAM>(at_row<const T>(a.dy, row, a.ld_dy, from[k]), N);
      v.h[k] = load_vec<T, STREAM>(at_row<const T>(a.h, row, a.ld_h, from[k]), N);
      v.dh[k] = load_vec<T, STREAM>(at_row<const T>(dh, row, ld_dh, from[k]), N);
      v.x[k] = load_vec<T, STREAM>(at_row<const T>(a.x, row, a.ld_x, from[k]), N);
      if constexpr (TOKEN) v.gate[k] = load_vec<T, STREAM>(at_row<const T>(a.gate, row, a.ld_gate, from[k]), N);
    }
  };
  const uint32_t step = gridDim.x * groups;
  const float per_col = 1.0f / (float)a.cols;
  NormsRow<VPT> next;
  if constexpr (AHEAD) load(blockIdx.x * groups, next);
#pragma unroll 2
  for (uint32_t c = threadIdx.x * 4; c < width; c += blockDim.x * 4) {
    const int n = inside<4>(c, a.cols);
    float pre[4] = {}, post[4] = {}, gate[4] = {};
    if (n > 0) {
      load_gamma<4>(a.pre, a.gamma_f32, c, n, pre);
      load_gamma<4>(a.post, a.gamma_f32, c, n, post);
      if constexpr (KIND == kChannel) load_gamma<4>(a.gate, sizeof(T) == 4, c, n, gate);
    }
    *reinterpret_cast<u32x4_t*>(gains + c) = VecOf<float>::pack(pre);
    *reinterpret_cast<u32x4_t*>(gains + width + c) = VecOf<float>::pack(post);
    if constexpr (KIND == kChannel) {
#pragma unroll
      for (int i = 0; i < 4; i++) gate[i] = a.sigmoid ? sigmoid(gate[i]) : gate[i];
      *reinterpret_cast<u32x4_t*>(gains + 2 * width + c) = VecOf<float>::pack(gate);
    }
  }
  __syncthreads();
  for (uint32_t r0 = blockIdx.x * groups; r0 < a.rows; r0 += step) {
    const uint32_t row = r0 + grp;
    NormsRow<VPT> v;
    if constexpr (AHEAD) {
      v = next;
      load(r0 + step, next);  // at most 2^28 rows, and 2^20 to a step
    } else {
      load(r0, v);
    }
#pragma unroll
    for (int k = 0; k < VPT; k++)
      if (sh[k] != 0 || row >= a.rows) {
        const int by = row < a.rows ? sh[k] : N;
        shift_down<T>(v.dy[k], by);
        shift_down<T>(v.h[k], by);
        shift_down<T>(v.dh[k], by);
        shift_down<T>(v.x[k], by);
        if constexpr (TOKEN) shift_down<T>(v.gate[k], by);
      }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
#pragma unroll
      for (int u = 0; u < N / 4; u++) {
        float dy[4], nh[4], gm[4];
        unpack_four<T>(v.dy[k], u, dy);
        unpack_four<T>(v.h[k], u, nh);
        lds_four(gains + (j + k * G) * N + 4 * u, gm);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          nh[i] *= v.pre;
          s = __builtin_fmaf(dy[i] * gm[i], nh[i], s);
          acc_pre[k][4 * u + i] = __builtin_fmaf(dy[i], nh[i], acc_pre[k][4 * u + i]);
        }
      }
      packed(v.dy[k]);
      packed(v.h[k]);
      added(acc_pre[k]);
    }
    const float mean_pre = group_sum_once(s, G, red[0]) * per_col;
    float b[VPT][N];
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const uint32_t c = (j + k * G) * N;
      const int n = row < a.rows ? N - sh[k] : 0;
      u32x4_t out_r, out_g;
      opaque(to[k]);
#pragma unroll
      for (int u = 0; u < N / 4; u++) {
        float dy[4], h[4], gm[4], t[4], m[4], gate[4], dg[4];
        const u32x4_t vdh = v.dh[k] & dh_mask;
        unpack_four<T>(v.dy[k], u, dy);
        unpack_four<T>(v.h[k], u, h);
        unpack_four<T>(vdh, u, t);
        lds_four(gains + c + 4 * u, gm);
        back_vec<4>(t, dy, h, gm, v.pre, mean_pre);
        pack_four<T>(out_r, u, t);
        unpack_four<T>(v.x[k], u, m);
        lds_four(gains + width + c + 4 * u, gm);
        if constexpr (TOKEN) unpack_four<T>(v.gate[k], u, gate);
        if constexpr (KIND == kChannel) lds_four(gains + 2 * width + c + 4 * u, gate);
#pragma unroll
        for (int i = 0; i < 4; i++) m[i] *= v.post;
        gate_vec<KIND, 4>(a.scale, t, m, gate, gm, &b[k][4 * u], &acc_post[k][4 * u], dg);
        if constexpr (TOKEN) pack_four<T>(out_g, u, dg);
#pragma unroll
        for (int i = 0; i < 4; i++) s = __builtin_fmaf(b[k][4 * u + i], m[i], s);
      }
      packed(v.x[k]);
      added(acc_post[k]);
      if (n > 0 && a.dr != nullptr) store_vec<T, STREAM>(at_row<T>(a.dr, row, a.ld_dr, to[k]), out_r, n);
      if constexpr (TOKEN)
        if (n > 0 && a.dgate != nullptr) store_vec<T, STREAM>(at_row<T>(a.dgate, row, a.ld_dgate, to[k]), out_g, n);
    }
    const float f = -(v.post * (group_sum_once(s, G, red[1]) * per_col));
    if (a.dx == nullptr) continue;
#pragma unroll
    for (int k = 0; k < VPT; k++) {
      const int n = row < a.rows ? N - sh[k] : 0;
      float m[N];
      VecOf<T>::unpack(v.x[k], m);
#pragma unroll
      for (int i = 0; i < N; i++) m[i] = v.post * __builtin_fmaf(m[i], f, b[k][i]);
      if (n > 0) store_vec<T, STREAM>(at_row<T>(a.dx, row, a.ld_dx, to[k]), VecOf<T>::pack(m), n);
    }
  }
  auto leave = [&](const float (&acc)[VPT][N], float* part) {
    if (part == nullptr) return;
    float* out = part + (int64_t)blockIdx.x * a.cols;
    if (groups == 1) {
#pragma unroll
      for (int k = 0; k < VPT; k++)
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const uint32_t c = (j + k * G) * N + i;
          if (c < a.cols) store_vec<float>(out + c, VecOf<float>::pack(&acc[k][i]), (int)(a.cols - c));
        }
      return;
    }
    __syncthreads();  // the gains, or the other sums, are read
    for (int q = 0; q < groups; q++) {
      if (grp == q) {
#pragma unroll
        for (int k = 0; k < VPT; k++)
#pragma unroll
          for (int i = 0; i < N; i++) {
            float* p = gains + (j + k * G) * N + i;
            *p = q == 0 ? acc[k][i] : *p + acc[k][i];
          }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += blockDim.x) out[c] = gains[c];
  };
  leave(acc_pre, a.pre_part);
  leave(acc_post, a.post_part);
}

// Wider rows: one workgroup a row at a time, read for each of its two sums and for its
// outputs; the column sums stay in the workgroup's rows of the workspace (each lane adds
// to its own columns).
template <typename T, int KIND>
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
    // t, m, b, d * m (added to sum) and dgate of one vector
    auto form = [&](uint64_t c, float* t, float* m, float* b, float* sum, float* dg) {
      const int n = inside<N>(c, a.cols);
      float dy[N], h[N], gm[N];
      at(a.dy, a.ld_dy, c, dy);
      at(a.h, a.ld_h, c, h);
      at(a.dh, a.ld_dh, c, t);
      at(a.x, a.ld_x, c, m);
      load_gamma<N>(a.pre, a.gamma_f32, (uint32_t)c, n, gm);
      back_vec<N>(t, dy, h, gm, pre, mean_pre);
      load_gamma<N>(a.post, a.gamma_f32, (uint32_t)c, n, gm);
#pragma unroll
      for (int i = 0; i < N; i++) m[i] *= post;
      float gate[N];
      if constexpr (KIND != kNoGate) at(a.gate, a.ld_gate, c, gate);
      if constexpr (KIND == kChannel)
#pragma unroll
        for (int i = 0; i < N; i++) gate[i] = a.sigmoid ? sigmoid(gate[i]) : gate[i];
      gate_vec<KIND, N>(a.scale, t, m, gate, gm, b, sum, dg);
    };
    s = 0.0f;
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      float t[N], m[N], b[N], sum[N] = {}, dg[N], q = 0.0f;
      form(c, t, m, b, sum, dg);
#pragma unroll
      for (int i = 0; i < N; i++) q = __builtin_fmaf(b[i], m[i], q);
      s += q;
    }
    const float mean_post = group_sum(s, 1024, red) / (float)a.cols;
    for (uint64_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {
      const int n = inside<N>(c, a.cols);
      float t[N], m[N], b[N], sum[N] = {}, dg[N], dy[N], h[N];
      form(c, t, m, b, sum, dg);
      at(a.dy, a.ld_dy, c, dy);
      at(a.h, a.ld_h, c, h);
      const bool first = row == blockIdx.x;
#pragma unroll
      for (int i = 0; i < N; i++) {
        if (i >= n) continue;
        if (out_pre != nullptr) out_pre[c + i] = __builtin_fmaf(dy[i], h[i] * pre, first ? 0.0f : out_pre[c + i]);
        if (out_post != nullptr) out_post[c + i] = sum[i] + (first ? 0.0f : out_post[c + i]);
      }
#pragma unroll
      for (int i = 0; i < N; i++) m[i] = post * __builtin_fmaf(-m[i], mean_post, b[i]);
      if (a.dr != nullptr) store_vec(static_cast<T*>(a.dr) + (int64_t)row * a.ld_dr + c, VecOf<T>::pack(t), n);
      if constexpr (KIND != kNoGate && KIND != kChannel)
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
  // Beyond the registers, or less than a vector: a workgroup for each row, which narrow rows in number
  // pay for (2^20 x 4 BF16 39 ms; x 8, in registers, 0.18).
  if (b.row.vpt * N > 16 || cols < N) b.row = RowShape{0, 0};
  if (b.row.vpt == 0) return BackShape{b.row, 1, std::min<int64_t>(rows, kCus)};
  // As many rows as a workgroup of 1024 lanes takes share a copy of the gains and a row of
  // sums, while that leaves a workgroup to each CU (16384 x 4096 BF16 with a gate per row
  // 188 us, 202 with 512 lanes; 300 x 2048 without 11.0, and 11.6 with four rows).  Groups of a
  // wave or less meet no barrier, and add their sums one after the other: 256 lanes
  // (16384 x 200 19.4 us, 21.7 with 512, 24.5 with 1024).
  b.groups = (int)std::min<int64_t>(std::max(1, (b.row.G <= 64 ? 256 : 1024) / b.row.G), (rows + kCus - 1) / kCus);
  // the workgroups that a CU holds, by their registers: two of up to eight waves (twelve
  // where a lane has four elements), or one
  const int threads = b.row.G * b.groups;
  const bool two = threads <= (b.row.vpt * N <= 4 ? 768 : 512);
  b.parts = std::min((rows + b.groups - 1) / b.groups, two ? 2 * kCus : kCus);
  return b;
}

// LDS of the backward pass's gains at most: beside it the workgroup's sums, within 160 KB.
constexpr int kMostGains = 150 * 1024;

template <typename T, int KIND>
hipError_t norms_back_t(const NormsBackArgs& a, const BackShape& b, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  // the gains, and a gate that is one row for all; the groups' sums meet there
  const int64_t lds = (int64_t)b.row.G * b.row.vpt * N * (KIND == kChannel ? 12 : 8);
  if (b.row.vpt == 0 || lds > kMostGains) {
    k_block_norms_back_wide<T, KIND><<<(unsigned)b.parts, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const bool stream = (int64_t)a.rows * a.cols * 6 * (int64_t)sizeof(T) >= kStreamBytes;
  hipError_t e = hipSuccess;
  with_vpt(b.row.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value * N <= 16 ? vpt.value : 1;  // what back_shape picks
    auto* kernel = stream ? &k_block_norms_back<T, VPT, KIND, true, true> : &k_block_norms_back<T, VPT, KIND, false, true>;
    if constexpr (VPT == 1)
      if (b.row.G < 64) kernel = &k_block_norms_back<T, 1, KIND, false, false>;
    if (lds > 64 * 1024) {
      static std::atomic<uint64_t> done{0};
      e = allow_lds(done, kMostGains, &k_block_norms_back<T, VPT, KIND, true, true>,
                    &k_block_norms_back<T, VPT, KIND, false, true>);
    }
    if (e == hipSuccess) kernel<<<(unsigned)b.parts, b.groups * b.row.G, lds, s>>>(a, b.row.G);
  });
  return e == hipSuccess ? hipGetLastError() : e;
}
template <typename T>
hipError_t norms_back_kind(const NormsBackArgs& a, const BackShape& b, bool shared, hipStream_t s) {
  if (a.gate == nullptr) return norms_back_t<T, kNoGate>(a, b, s);
  if (shared) return norms_back_t<T, kChannel>(a, b, s);
  return a.sigmoid ? norms_back_t<T, kTokenSigmoid>(a, b, s) : norms_back_t<T, kToken>(a, b, s);
}

template <typename T, bool CODES>
hipError_t norms_t(const NormsArgs& a, hipStream_t s) {
  constexpr int N = VecOf<T>::N;
  const int64_t vecs = ((CODES ? (int64_t)a.padded : (int64_t)a.cols) + N - 1) / N;
  // Two vectors a lane and half the waves where rows are many (BF16 with a gate per row: 8192 x
  // 5120 68 us, 79 with one, 68 with three; 32768 x 1024 54, 59, 55; 32768 x 256 19 and 21).  One where
  // a launch is as long as its longest row (48 x 5120 4.5 us, 4.7 with two), and up to the 16 vectors
  // that a group has lanes for (32768 x 128 12.0, 13.2 with two).
  const RowShape r = row_shape(vecs, a.rows >= 512 && vecs > 16 ? 2 : 1);
  if (r.vpt == 0 || r.vpt > 5) {
    k_block_norms_wide<T, CODES><<<a.rows, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const int threads = r.G < 64 ? 256 / r.G * r.G : r.G;
  const unsigned grid = (a.rows + threads / r.G - 1) / (threads / r.G);
  const bool stream = (int64_t)a.rows * a.cols * 4 * (int64_t)sizeof(T) >= kStreamBytes;
  with_vpt(r.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value <= 5 ? vpt.value : 1;
    auto* kernel = a.cols % N == 0
                       ? stream ? &k_block_norms<T, VPT, CODES, true, true> : &k_block_norms<T, VPT, CODES, false, true>
                   : stream ? &k_block_norms<T, VPT, CODES, true, false>
                            : &k_block_norms<T, VPT, CODES, false, false>;
    kernel<<<grid, threads, 0, s>>>(a, r.G);
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
                          gamma_dt,  gate_act,  scale};
    const hipError_t e = dt == 0 ? norms_back_kind<uint16_t>(a, b, shared, s) : norms_back_kind<float>(a, b, shared, s);
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
