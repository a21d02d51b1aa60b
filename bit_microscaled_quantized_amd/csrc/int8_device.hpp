// Device pieces of the product of 8-bit integers (int8_gemm.hip, int8_few.hip): its
// arguments, and the scaled output of four sums in a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.hpp"

namespace nvfp4 {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx16 __attribute__((ext_vector_type(16)));

struct GemmArgs {
  const int8_t* a;
  const int8_t* b;
  const float* a_scales;
  const float* b_scales;
  void* c;
  int* partial;  // the parts' sums; null: no parts
  int64_t lda, ldb, ldc;
  int M, N, K;
  int whole;  // tiles taken whole (int8_gemm.hip); the rest, and every block of int8_few.hip, in parts
  int parts;
};

typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4), may_alias));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2), may_alias));

// Four output columns from n on of row m.
template <typename OutT>
__device__ __forceinline__ void store_four(const GemmArgs& g, int m, int n, const intx4& v, const float* bs, float as) {
  float f[4];
#pragma unroll
  for (int e = 0; e < 4; e++) f[e] = ((float)v[e] * bs[e]) * as;
  OutT* p = static_cast<OutT*>(g.c) + (int64_t)m * g.ldc + n;
  if (n + 4 <= g.N) {
    if constexpr (sizeof(OutT) == 4)
      *reinterpret_cast<f32x4_a4*>(p) = f32x4_a4{f[0], f[1], f[2], f[3]};
    else
      *reinterpret_cast<u32x2_a2*>(p) = u32x2_a2{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (n + e < g.N) {
      if constexpr (sizeof(OutT) == 4)
        p[e] = f[e];
      else
        p[e] = (uint16_t)bf16_pack(f[e], 0.0f);
    }
}

// Scales of four columns from n on (zeros past the last).
__device__ __forceinline__ void four_scales(const GemmArgs& g, int n, float* bs) {
#pragma unroll
  for (int e = 0; e < 4; e++) bs[e] = n + e < g.N ? g.b_scales[n + e] : 0.0f;
}

// The product for up to 64 tokens (int8_few.hip): parts of K, and bytes of workspace.
struct FewPlan {
  int parts;
  int64_t bytes;
};
FewPlan few_plan(int64_t M, int64_t N, int64_t K);
hipError_t int8_few(const GemmArgs& g, int c_dt, hipStream_t s);

}  // namespace nvfp4
