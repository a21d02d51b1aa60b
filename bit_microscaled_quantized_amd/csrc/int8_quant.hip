// Codes and scale of each row of a tensor, or of a gated activation
// (nvfp4_int8_quantize, nvfp4_int8_quantize_gated), for gfx950.
//
// Bound by HBM: a group of lanes holds a row in registers between its largest
// magnitude and its codes, so each input is read once; rows wider than a
// workgroup's registers are read (and the activation formed) twice.  8192 x 5120 BF16:
// 126 MB in 24 us (5.2 TB/s) over tensors that change from call to call; 20 over the same ones, which
// the caches hold in part, and 28 to 30 between two products of 8192 tokens.
#include "act_device.hpp"
#include "blocks_launch.hpp"
#include "row_codes.hpp"

namespace nvfp4 {

namespace {

struct QuantArgs {
  const void* gate;
  const void* up;
  int8_t* codes;
  float* scales;
  int64_t ld_g, ld_u, ld_codes;
  uint32_t rows, cols, padded;  // padded: cols up to a multiple of 16
};

// v of a vector's elements
template <typename T, int ACT>
__device__ __forceinline__ void values_of(const QuantArgs& a, u32x4_t g, u32x4_t u, float* f) {
  constexpr int N = VecOf<T>::N;
  float fu[N];
  VecOf<T>::unpack(g, f);
  VecOf<T>::unpack(u, fu);
#pragma unroll
  for (int i = 0; i < N; i++) {
    f[i] = act_of<ACT>(f[i]);
    if (a.up != nullptr) f[i] *= fu[i];
  }
}

template <typename T, int ACT, int VPT, bool STREAM>
__global__ __launch_bounds__(1024) void k_int8_rows(QuantArgs a, int G) {
  constexpr int N = VecOf<T>::N;
  __shared__ uint32_t red[16];
  const uint32_t row = blockIdx.x * (blockDim.x / G) + threadIdx.x / G, j = threadIdx.x % G;
  const bool live = row < a.rows;
  const T* gr = static_cast<const T*>(a.gate) + (int64_t)row * a.ld_g;
  const T* ur = static_cast<const T*>(a.up) + (int64_t)row * a.ld_u;
  u32x4_t g[VPT], u[VPT];
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live && c < a.cols ? (int)min(a.cols - c, (uint32_t)N) : 0;
    g[k] = load_row<T, STREAM, false>(gr, c, n, a.cols);
    u[k] = load_row<T, STREAM, false>(ur, c, a.up == nullptr ? 0 : n, a.cols);
  }
  float f[VPT][N];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    const int n = live && c < a.cols ? (int)min(a.cols - c, (uint32_t)N) : 0;
    end_row<T>(g[k], n, a.cols);
    end_row<T>(u[k], n, a.cols);
    values_of<T, ACT>(a, g[k], u[k], f[k]);  // zeros past the row's end
    m = most_of<N>(f[k], m);
  }
  const RowCode q(group_max(m, G, red));
  if (!live) return;
  if (j == 0) a.scales[row] = q.scale;
  int8_t* out = a.codes + (int64_t)row * a.ld_codes;
#pragma unroll
  for (int k = 0; k < VPT; k++) {
    const uint32_t c = (j + k * G) * N;
    if (c < a.padded) store_codes<N>(q, f[k], out, c);
  }
}

// Wider rows: one workgroup a row.
template <typename T, int ACT>
__global__ __launch_bounds__(1024) void k_int8_wide(QuantArgs a) {
  constexpr int N = VecOf<T>::N;
  __shared__ uint32_t red[16];
  const uint32_t row = blockIdx.x;
  const T* gr = static_cast<const T*>(a.gate) + (int64_t)row * a.ld_g;
  const T* ur = static_cast<const T*>(a.up) + (int64_t)row * a.ld_u;
  auto at = [&](uint32_t c, float* f) {
    const int n = c < a.cols ? (int)min(a.cols - c, (uint32_t)N) : 0;
    values_of<T, ACT>(a, load_or_zero<T, false>(gr, c, n, a.cols),
                      load_or_zero<T, false>(ur, c, a.up == nullptr ? 0 : n, a.cols), f);
  };
  uint32_t m = 0;
  for (uint32_t c = threadIdx.x * N; c < a.cols; c += 1024 * N) {  // fewer than 2^31 columns
    float f[N];
    at(c, f);
    m = most_of<N>(f, m);
  }
  const RowCode q(group_max(m, 1024, red));
  if (threadIdx.x == 0) a.scales[row] = q.scale;
  int8_t* out = a.codes + (int64_t)row * a.ld_codes;
  for (uint32_t c = threadIdx.x * N; c < a.padded; c += 1024 * N) {
    float f[N];
    at(c, f);
    store_codes<N>(q, f, out, c);
  }
}

// Vectors a lane: one finishes a few rows soonest, two or (wide rows) five stream best, over tensors that
// change (8192 x 5120 bf16 36.0 us with one, 24.1 with two, 24.0 with five; 4096 x 5120 fp32 22.0,
// 22.1, 21.4; 2048 x 4096 bf16 8.1, 7.4, 7.7; 300 x 5120 4.5, 5.0, 4.7) as over the same ones (27.8, 20.5,
// 20.3; 18.1, 18.4, 16.5; 6.5, 5.5, 5.6; 4.7, 4.6, 4.6).
template <typename T, int ACT>
hipError_t quantize_t(const QuantArgs& a, hipStream_t s) {
  const int64_t vecs = a.padded / VecOf<T>::N;
  const RowShape r = row_shape(vecs, a.rows < 1024 || vecs <= 128 ? 1 : vecs <= 512 ? 2 : 5);
  if (r.vpt == 0 || r.vpt > 5) {
    k_int8_wide<T, ACT><<<a.rows, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const int threads = r.G < 64 ? 256 / r.G * r.G : r.G;
  const unsigned grid = (a.rows + threads / r.G - 1) / (threads / r.G);
  const bool stream = (int64_t)a.rows * a.cols * (int64_t)sizeof(T) * (a.up == nullptr ? 1 : 2) >= kStreamBytes;
  with_vpt(r.vpt, [&](auto vpt) {
    constexpr int VPT = vpt.value <= 5 ? vpt.value : 1;
    if (stream)
      k_int8_rows<T, ACT, VPT, true><<<grid, threads, 0, s>>>(a, r.G);
    else
      k_int8_rows<T, ACT, VPT, false><<<grid, threads, 0, s>>>(a, r.G);
  });
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                                int64_t ld_g, int64_t ld_u, int8_t* codes, int64_t ld_codes, float* scales,
                                hipStream_t s) {
  const QuantArgs a{gate, up,       codes,          scales,         ld_g,
                    ld_u, ld_codes, (uint32_t)rows, (uint32_t)cols, (uint32_t)((cols + 15) / 16 * 16)};
  hipError_t e = hipSuccess;
  with_act(act, [&](auto kind) {
    e = dt == 0 ? quantize_t<uint16_t, kind.value>(a, s) : quantize_t<float, kind.value>(a, s);
  });
  return e;
}

}  // namespace nvfp4
