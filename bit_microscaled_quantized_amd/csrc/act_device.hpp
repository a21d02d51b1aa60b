// Device pieces of the gated activation (activation.hip) and of the quantization
// behind it (int8_quant.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.hpp"

namespace nvfp4 {

constexpr float kLog2e_act = 1.44269504088896340736f;

// 1 / (1 + exp(-v)) by the hardware's 2^x and reciprocal: within 4 u + 2 |v| u, u = 2^-24
// (the exponent's rounding, the instructions' 1 ulp each, the sum's).
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e_act));
}

enum Act { kNone = 0, kSilu = 1, kGelu = 2, kRelu2 = 3 };

// act(v); with SLOPE its derivative as well.  GELU's (1 + tanh t) / 2 is the logistic
// function p of 2 t; where v^2 overflows its slope is p, whose other term holds 1 - p or a
// of 0: v^2 is bounded, so that the term is 0 and not 0 times infinity.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float act_of(float v, float& slope) {
  if constexpr (ACT == kSilu) {
    const float p = sigmoid(v), a = v * p;
    if constexpr (SLOPE) slope = __builtin_fmaf(a, 1.0f - p, p);
    return a;
  } else if constexpr (ACT == kGelu) {
    constexpr float C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float q = v * v;
    const float p = sigmoid(v * __builtin_fmaf(q, C * 0.044715f, C)), a = v * p;
    if constexpr (SLOPE)
      slope = __builtin_fmaf(a * (1.0f - p), __builtin_fmaf(fminf(q, 1e30f), 3.0f * C * 0.044715f, C), p);
    return a;
  } else if constexpr (ACT == kRelu2) {
    const float r = v < 0.0f ? 0.0f : v;  // NaN stays
    if constexpr (SLOPE) slope = r + r;
    return r * r;
  } else {
    if constexpr (SLOPE) slope = 1.0f;
    return v;
  }
}
template <int ACT>
__device__ __forceinline__ float act_of(float v) {
  float unused;
  return act_of<ACT, false>(v, unused);
}

// f(ACT) with the activation as a constant
template <typename F>
void with_act(int act, F&& f) {
  using std::integral_constant;
  switch (act) {
    case kNone: f(integral_constant<int, kNone>{}); break;
    case kSilu: f(integral_constant<int, kSilu>{}); break;
    case kGelu: f(integral_constant<int, kGelu>{}); break;
    default: f(integral_constant<int, kRelu2>{});
  }
}

// A vector of a row (n of its elements inside it, n <= 0: none; the rest zero).
template <typename T, bool STREAM>
__device__ __forceinline__ u32x4_t load_or_zero(const T* p, int n) {
  return n > 0 ? load_vec<T, STREAM>(p, n) : u32x4_t{0, 0, 0, 0};
}

// The low bytes of four integers held as 1.5 * 2^23 + integer, in order.
__device__ __forceinline__ uint32_t bytes_of(float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000C0Cu);
  return lo | hi;
}
// Added to a number below 2^22 in magnitude, leaves its nearest even integer in the low bits.
constexpr float kToInt = 12582912.0f;

}  // namespace nvfp4
