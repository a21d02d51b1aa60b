// Device pieces of the gated activation (activation.hip) and of the quantization
// behind it (int8_quant.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.hpp"

namespace nvfp4 {

constexpr float kLog2e_act = 1.44269504088896340736f;

// 1 / (1 + exp(-v)) by the hardware's 2^x and reciprocal: within (5 + 1.25 |v|) u of itself, u = 2^-24 (the
// exponent's product by a rounded log2 e, the instructions' 1 ulp each, the sum's), where it is 2^-126
// or more.  Below, for v < -87.3, it is 0: the reciprocal has no subnormal results.
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

// A vector's elements from the sh-th on, zeros behind them.
template <typename T>
__device__ __forceinline__ void shift_down(u32x4_t& v, int sh) {
  const int words = sizeof(T) == 4 ? sh : sh >> 1;
  if (words & 4) v = u32x4_t{0, 0, 0, 0};
  if (words & 2) v = u32x4_t{v[2], v[3], 0, 0};
  if (words & 1) v = u32x4_t{v[1], v[2], v[3], 0};
  if (sizeof(T) == 2 && (sh & 1))
    v = u32x4_t{__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
                __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16};
}

// A row's vector from column c on (n of its elements inside it, n <= 0: none).  One that
// ends past the row is read as the row's last whole one, for end_row to shift when all of a
// lane's loads are under way (8192 x 5119 BF16 norms 91 us; with its elements read one after
// the other 132).  WHOLE: none does.
template <typename T, bool STREAM, bool WHOLE, typename I>
__device__ __forceinline__ u32x4_t load_row(const T* row, I c, int n, uint32_t cols) {
  constexpr int N = VecOf<T>::N;
  if (n <= 0) return u32x4_t{0, 0, 0, 0};
  if constexpr (WHOLE) return load_vec<T, STREAM>(row + c, N);
  if (cols < (uint32_t)N) return VecOf<T>::load_n(row, n);
  return load_vec<T, STREAM>(row + min(c, (I)(cols - N)), N);
}
// The rest of its elements zero.
template <typename T>
__device__ __forceinline__ void end_row(u32x4_t& v, int n, uint32_t cols) {
  constexpr int N = VecOf<T>::N;
  if (n > 0 && n < N && cols >= (uint32_t)N) shift_down<T>(v, N - n);
}
// Both
template <typename T, bool STREAM, typename I>
__device__ __forceinline__ u32x4_t load_or_zero(const T* row, I c, int n, uint32_t cols) {
  u32x4_t v = load_row<T, STREAM, false>(row, c, n, cols);
  end_row<T>(v, n, cols);
  return v;
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
