// Codes of a row with one scale (int8_quant.hip, block_norms.hip): the row's largest
// magnitude gives the factor, codes leave as bytes, zeros up to a multiple of 16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act_device.hpp"
#include "rows_device.hpp"

namespace nvfp4 {

namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}

// Largest over the aligned 16, 32 or 64 lanes of a span (span_sum's butterfly).
__device__ __forceinline__ uint32_t span_max(uint32_t v, int span) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  v = dpp_max<0x140>(v);
  if (span > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  if (span > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  return v;
}

// Largest over the G lanes of a group (group_sum's way; every lane of the workgroup).
__device__ __forceinline__ uint32_t group_max(uint32_t v, int G, uint32_t* red) {
  v = span_max(v, G);
  if (G > 64) {
    __syncthreads();  // the last use of red is over
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = G / 64, first = (int)threadIdx.x / G * waves, w = threadIdx.x & 15;
    v = span_max(w >= first && w < first + waves ? red[w] : 0u, 16);
  }
  return v;
}

// A row's factor and scale from the bits of its largest magnitude.
struct RowCode {
  float inv, scale;
  bool zero;  // codes are 0 whatever the values (an infinity or a NaN among them)
  __device__ __forceinline__ explicit RowCode(uint32_t most) {
    const float amax = __uint_as_float(most);
    zero = most >= 0x7F800000u;
    const bool live = !zero && amax >= 0x1p-100f;
    inv = live ? 127.0f / amax : 0.0f;
    scale = zero ? __builtin_nanf("") : live ? amax / 127.0f : 0.0f;
  }
  __device__ __forceinline__ uint32_t four(const float* f) const {
    const uint32_t w = bytes_of(f[0] * inv + kToInt, f[1] * inv + kToInt, f[2] * inv + kToInt, f[3] * inv + kToInt);
    return zero ? 0u : w;
  }
};

// Largest magnitude of N values, on the bits.
template <int N>
__device__ __forceinline__ uint32_t most_of(const float* f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < N; i++) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

// Codes of the N (4 or 8) values from column c on, which are zeros past the row's end:
// whole pieces, as rows of codes are multiples of 16 bytes.
template <int N>
__device__ __forceinline__ void store_codes(const RowCode& q, const float* f, int8_t* row, uint32_t c) {
  if constexpr (N == 8)
    *reinterpret_cast<u32x2_t*>(row + c) = u32x2_t{q.four(f), q.four(f + 4)};
  else
    *reinterpret_cast<uint32_t*>(row + c) = q.four(f);
}

}  // namespace

}  // namespace nvfp4
