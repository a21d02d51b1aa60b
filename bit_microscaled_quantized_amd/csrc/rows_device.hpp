// Kernels that hold rows in registers (norm.hip, block_norms.hip, int8_quant.hip):
// sums and maxima over a group of lanes that shares a row, a row's gains, and how
// many lanes and vectors a lane a row takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "layers_device.hpp"

namespace nvfp4 {

namespace {

// v of another lane of its 16: DPP control CTRL
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// Sum over the aligned 16, 32 or 64 lanes of a span, a butterfly in the registers:
// neighbours, pairs, quads (half mirrored), halves of 16 (mirrored), rows of 16,
// halves of the wave.  (Through LDS, shuffle by shuffle, a sum over a wave takes
// some 500 cycles, a tenth of what a row of 5120 takes in all.)
__device__ __forceinline__ float span_sum(float v, int span) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  if (span > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (span > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Sum over the G lanes of a group: inside a wave, or through the group's G / 64
// places in red, one per wave of the workgroup; every lane gets the result.  All
// lanes of the workgroup call it together.
__device__ __forceinline__ float group_sum(float v, int G, float* red) {
  v = span_sum(v, G);
  if (G > 64) {
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = G / 64, first = (int)threadIdx.x / G * waves, w = threadIdx.x & 15;
    v = span_sum(w >= first && w < first + waves ? red[w] : 0.0f, 16);
  }
  return v;
}

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

// Lanes and vectors per lane of a row of `vecs` vectors, with `want` vectors a lane
// where up to 1024 lanes allow it; vpt 0 where the row is too wide.
struct RowShape {
  int G, vpt;
};
RowShape row_shape(int64_t vecs, int want) {
  for (int vpt : {1, 2, 3, 5, 8}) {
    if (vpt < want || vecs > 1024 * vpt) continue;
    const int lanes = (int)((vecs + vpt - 1) / vpt);
    return RowShape{lanes <= 16 ? 16 : lanes <= 32 ? 32 : (lanes + 63) / 64 * 64, vpt};
  }
  return RowShape{0, 0};
}

// f(VPT) with the number of vectors as a constant
template <typename F>
void with_vpt(int vpt, F&& f) {
  using std::integral_constant;
  switch (vpt) {
    case 1: f(integral_constant<int, 1>{}); break;
    case 2: f(integral_constant<int, 2>{}); break;
    case 3: f(integral_constant<int, 3>{}); break;
    case 5: f(integral_constant<int, 5>{}); break;
    default: f(integral_constant<int, 8>{});
  }
}

}  // namespace

}  // namespace nvfp4
