// Device helpers of the operators between the quantized layers (norm.hip,
// loss.hip): 16-byte vectors of BF16 or FP32 at element alignment, and the
// dropout mask from the counter hash.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_device.hpp"

namespace nvfp4 {

// 16-byte vectors that need only their element's alignment (rows of an odd
// width start anywhere): gfx950 loads and stores them in one instruction.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4), may_alias));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1), may_alias));
typedef uint32_t u32_a1 __attribute__((aligned(1), may_alias));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));

// Two FP32 values to BF16, nearest even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t bf16_pack(float a, float b) {
  const bf16x2_t v = __builtin_convertvector((floatx2_t{a, b}), bf16x2_t);
  return __builtin_bit_cast(uint32_t, v);
}

// Element type of a tensor: float, or uint16_t for BF16 bits.
template <typename T>
struct VecOf;

template <>
struct VecOf<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ u32x4_t load(const uint16_t* p) { return *reinterpret_cast<const u32x4_a2*>(p); }
  static __device__ __forceinline__ void store(uint16_t* p, u32x4_t v) { *reinterpret_cast<u32x4_a2*>(p) = v; }
  static __device__ __forceinline__ u32x4_t load_nt(const uint16_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
  }
  static __device__ __forceinline__ void store_nt(uint16_t* p, u32x4_t v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(p));
  }
  // the first n < 8 elements, the rest zero
  static __device__ __forceinline__ u32x4_t load_n(const uint16_t* p, int n) {
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return v;
  }
  static __device__ __forceinline__ void store_n(uint16_t* p, u32x4_t v, int n) {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
  static __device__ __forceinline__ void unpack(u32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      f[2 * i] = bf16lo(v[i]);
      f[2 * i + 1] = bf16hi(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{bf16_pack(f[0], f[1]), bf16_pack(f[2], f[3]), bf16_pack(f[4], f[5]), bf16_pack(f[6], f[7])};
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
};

template <>
struct VecOf<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ u32x4_t load(const float* p) { return *reinterpret_cast<const u32x4_a4*>(p); }
  static __device__ __forceinline__ void store(float* p, u32x4_t v) { *reinterpret_cast<u32x4_a4*>(p) = v; }
  static __device__ __forceinline__ u32x4_t load_nt(const float* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a4*>(p));
  }
  static __device__ __forceinline__ void store_nt(float* p, u32x4_t v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a4*>(p));
  }
  static __device__ __forceinline__ u32x4_t load_n(const float* p, int n) {
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < n) v[i] = __float_as_uint(p[i]);
    return v;
  }
  static __device__ __forceinline__ void store_n(float* p, u32x4_t v, int n) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < n) p[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ void unpack(u32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; i++) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

// n elements (n <= 0: none, n >= N: a whole vector) at p.  STREAM: past the caches.
template <typename T, bool STREAM = false>
__device__ __forceinline__ u32x4_t load_vec(const T* p, int n) {
  if (n >= VecOf<T>::N) return STREAM ? VecOf<T>::load_nt(p) : VecOf<T>::load(p);
  return VecOf<T>::load_n(p, n);
}
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_vec(T* p, u32x4_t v, int n) {
  if (n >= VecOf<T>::N)
    STREAM ? VecOf<T>::store_nt(p, v) : VecOf<T>::store(p, v);
  else
    VecOf<T>::store_n(p, v, n);
}

// Dropout of a call: the hash key of its seed, cut and the kept elements' factor.
struct Dropout {
  uint32_t key, cut;
  float scale;
};

inline Dropout make_dropout(float p, uint64_t seed) {
  Dropout d;
  d.key = sr_key(seed);
  d.cut = (uint32_t)__builtin_rint((double)p * 65536.0);
  d.scale = (float)(65536.0 / (65536.0 - (double)d.cut));
  return d;
}

// Dropout of N (4 or 8) consecutive elements from index i0: each hash word
// covers an even element (low half) and the odd one after it (high half).  Where
// i0 is a multiple of N the N / 2 pairs differ in their low bits only, which then
// come out of the hash's first product as a uniform term: one multiply for all.
template <int N>
__device__ __forceinline__ void drop(float* v, uint32_t i0, const Dropout& d) {
  constexpr uint32_t LOW = N / 2 - 1;
  const uint32_t pair = i0 >> 1;
  if ((i0 & (N - 1)) == 0) {
    uint32_t base = ((d.key ^ pair) & ~LOW) * 747796405u;
    asm volatile("" : "+v"(base));  // keep the shared product
#pragma unroll
    for (uint32_t q = 0; q < N / 2; q++) {
      const uint32_t h = pcg_tail(base + (((d.key & LOW) ^ q) * 747796405u + 2891336453u));
      v[2 * q] = (h & 0xFFFFu) >= d.cut ? v[2 * q] * d.scale : 0.0f;
      v[2 * q + 1] = (h >> 16) >= d.cut ? v[2 * q + 1] * d.scale : 0.0f;
    }
    return;
  }
  // an odd i0 starts with the high half of its pair
  uint32_t h = pcg_host(d.key ^ pair);
  const bool odd = (i0 & 1u) != 0;
#pragma unroll
  for (uint32_t q = 0; q < N / 2; q++) {
    uint32_t g = h;
    if (odd || q + 1 < N / 2) g = pcg_host(d.key ^ (pair + q + 1));
    const uint32_t b0 = odd ? h >> 16 : h & 0xFFFFu, b1 = odd ? g & 0xFFFFu : h >> 16;
    v[2 * q] = b0 >= d.cut ? v[2 * q] * d.scale : 0.0f;
    v[2 * q + 1] = b1 >= d.cut ? v[2 * q + 1] * d.scale : 0.0f;
    h = g;
  }
}

}  // namespace nvfp4
