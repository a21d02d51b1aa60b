// Device pieces shared by the kernels of the linear cross entropy (loss.hip,
// loss_few.hip), and the launcher of the latter.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "layers_device.hpp"

namespace nvfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

// exp(a): one multiply and the hardware's 2^x, within 1 ulp of exp(a (1 + e)), |e| <
// 2^-24 + 2^-26 (the product's rounding, and log2(e)'s to FP32); results below 2^-126
// are 0.
__device__ __forceinline__ float exp_fast(float a) { return __builtin_amdgcn_exp2f(a * kLog2e); }

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

// What the backward pass knows of its n[0] labelled tokens, in order: which
// tokens they are, and of every token its place among them (or -1).
//
// d is held in units of scale, the labelled tokens' largest |dloss|, which the
// results are multiplied by in FP32.  Tokens of a mean loss share one dloss; in its
// units a label that the model gives little is -1 and hardly rounded, where -dloss
// itself would be rounded alike for all tokens, up to 2^-8 of the whole gradient.
//
// One BF16 rounding of d, 2^-8 of it at most, averages out over a gradient's many
// terms, but a few tokens' gradients are one large term each (their labels'), and
// then it doubles the error of the result's own rounding.  Up to `half` labelled
// tokens d is therefore held in two parts, BF16 and the BF16 of what remains: token i
// takes columns i and half + i of d^T, rows i and half + i of xc.  The products'
// smallest tiles have the room, so this takes no longer.
struct Tokens {
  int* n;
  float* scale;
  int* place;
  int* list;
  int half;
  __device__ __forceinline__ bool two() const { return *n <= half; }
  // columns of d^T up to the last in use (those between the parts are zeros)
  __device__ __forceinline__ int columns() const { return *n == 0 ? 0 : two() ? half + *n : *n; }
};

// 16 aligned bytes; STREAM: past the caches, for a dw that they do not hold (257 x
// 49999 x 2048, 205 MB: 120 us for d and dw against 154; 69 x 14757 x 3160, 93 MB: 70
// against 61)
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, u32x4_t v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, static_cast<u32x4_t*>(p));
  else
    *static_cast<u32x4_t*>(p) = v;
}

// ---- the weight gradient of few tokens (loss_few.hip)

constexpr int FEW_DW_TOKENS = 32;

// dw (+)= dt^T xc for T <= FEW_DW_TOKENS; dt [rows][ldt] has zeros, and xc zero rows,
// past the last column up to a multiple of 32
hipError_t few_dw(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T, Tokens tk,
                  void* dw, int dw_f32, int64_t ld_dw, int accumulate, bool stream, hipStream_t s);

}  // namespace nvfp4
