// Device pieces shared by the kernels of the linear cross entropy (loss.hip for
// many tokens, loss_few.hip for few), and the launchers of the latter.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "layers_device.hpp"

namespace nvfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

// exp(a): one multiply and the hardware's 2^x, within 1 ulp of exp(a (1 + 2^-24));
// results below 2^-126 are 0.
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
struct Tokens {
  int* n;
  int* place;
  int* list;
};

// ---- up to 64 tokens (loss_few.hip)

constexpr int FEW_TOKENS = 64;
constexpr int FEW_ROWS = 32;       // vocabulary rows per workgroup of the logits kernels
constexpr int FEW_DW_TOKENS = 256;  // the dw kernel takes up to this many

// Tokens padded to 16, 32 or 64; columns of d^T.
inline int64_t few_tokens(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }
inline int64_t few_ldt(int64_t T) { return std::max<int64_t>(few_tokens(T), 32); }
inline int64_t few_rows(int64_t V) { return (V + FEW_ROWS - 1) / FEW_ROWS * FEW_ROWS; }
int64_t few_dx_parts(int64_t T, int64_t V, int64_t H);

// stats [T][few_rows(V) / FEW_ROWS], zlab [T]
hipError_t few_stats(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* x, uint32_t ld_x, int64_t T,
                     int64_t H, const int64_t* labels, float2* stats, float* zlab, hipStream_t s);
// dt [few_rows(V)][few_ldt(T)], d [few_tokens(T)][few_rows(V)]: zeros past the last token and row
hipError_t few_grad(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* xc, int64_t T, int64_t H, Tokens tk,
                    const int64_t* labels, const float* lse, const float* dloss, uint16_t* dt, uint16_t* d,
                    hipStream_t s);
// sum [parts][T][H]
hipError_t few_dx(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* d, int64_t T, int64_t H, Tokens tk,
                  float* sum, hipStream_t s);
// dw (+)= dt^T xc for T <= FEW_DW_TOKENS; dt has zeros, and xc zero rows, past the last token up to a multiple of 32
hipError_t few_dw(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T, Tokens tk,
                  void* dw, int dw_f32, int64_t ld_dw, int accumulate, hipStream_t s);

}  // namespace nvfp4
