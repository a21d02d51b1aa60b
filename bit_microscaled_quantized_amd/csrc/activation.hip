// The gated activation y = act(gate) * up whose inputs are kept in 8 bits, and its
// backward pass from them (nvfp4_gated_act, nvfp4_gated_act_backward), for gfx950.
//
// Both are bound by HBM: each element is read and written once, kept inputs one byte
// each and a scale byte per 32.  A lane takes 8 elements of a row (a block of 32 is
// four adjacent lanes); its block's largest magnitude goes through two lane swaps.
// A row's blocks are counted whole, so lanes past a ragged row's end have nothing
// to do but take part in those.
#include "act_device.hpp"
#include "blocks_launch.hpp"

namespace nvfp4 {

namespace {

// Quotients by a constant number of lanes a row, for any 32-bit numerator: with l =
// ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (m n / 2^32 + n) / 2^l,
// the sum halved first so that it stays in 32 bits (Granlund and Montgomery, 1994).
struct Divider {
  uint32_t d, m;
  int s1, s2;
};
Divider make_divider(uint32_t d) {
  int l = 0;
  while ((uint64_t(1) << l) < d) l++;
  const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1;
  return Divider{d, (uint32_t)m, l < 1 ? l : 1, l < 1 ? 0 : l - 1};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& v) {
  const uint32_t t = __umulhi(v.m, n);
  return (t + ((n - t) >> v.s1)) >> v.s2;
}

struct ActArgs {
  const void* gate;
  const void* up;
  void* y;
  int8_t* gate_codes;
  uint8_t* gate_scales;
  int8_t* up_codes;
  uint8_t* up_scales;
  int64_t ld_g, ld_u, ld_y;
  uint32_t items, cols, blocks;  // lanes' pieces of 8 elements in all; a row's elements and blocks
  Divider per_row;
};

// The larger of v and another lane's of the block of four lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}

// Codes and scale byte of a lane's eight elements; every lane of the block takes part.
__device__ __forceinline__ void keep(const float* f, uint32_t row, uint32_t c, int n, uint32_t cols,
                                     uint32_t blocks, int8_t* codes, uint8_t* scales) {
  // the largest magnitude, on the bits: infinities and NaN order above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = quad_max<0xB1>(m);
  m = quad_max<0x4E>(m);
  if (n <= 0) return;
  // m = a * 2^E, 1 <= a < 2: 127 = 1.984375 * 2^6, so the exponent is E - 6 for a <=
  // 1.984375 and E - 5 above.  A subnormal's E reads as -127, its limit for -133 is
  // 127 * 2^-133 = 0x7F0000 * 2^-149.
  const bool finite = m < 0x7F800000u;
  int e = (int)(m >> 23) - 127 - 6 + ((m & 0x7FFFFFu) > (m < 0x800000u ? 0x7F0000u : 0x7E0000u) ? 1 : 0);
  e = min(e, 121);
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; i++) t[i] = fminf(__builtin_amdgcn_ldexpf(f[i], -e), 127.0f) + kToInt;
  uint32_t w[2] = {bytes_of(t[0], t[1], t[2], t[3]), bytes_of(t[4], t[5], t[6], t[7])};
  if (!finite) w[0] = w[1] = 0;
  int8_t* p = codes + (int64_t)row * cols + c;
  if (n >= 8) {
    *reinterpret_cast<u32x2_a1*>(p) = u32x2_t{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < n) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if ((c & 31) == 0)
    scales[(int64_t)row * blocks + c / 32] = finite ? (uint8_t)(e + 133) : (uint8_t)255;
}

template <typename T, int ACT, bool STREAM>
__global__ __launch_bounds__(256) void k_act(ActArgs a) {
  const uint32_t item = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = divide(item, a.per_row), c = (item - row * a.per_row.d) * 8;
  const int n = item < a.items && c < a.cols ? (int)min(a.cols - c, 8u) : 0;
  Eight<T, STREAM> g, u;
  g.load(static_cast<const T*>(a.gate) + (int64_t)row * a.ld_g + c, n);
  if (a.up != nullptr) u.load(static_cast<const T*>(a.up) + (int64_t)row * a.ld_u + c, n);
  float fg[8], fu[8];
  g.unpack(fg);
  if (a.up != nullptr) u.unpack(fu);
  if (a.gate_codes != nullptr) {
    keep(fg, row, c, n, a.cols, a.blocks, a.gate_codes, a.gate_scales);
    if (a.up != nullptr) keep(fu, row, c, n, a.cols, a.blocks, a.up_codes, a.up_scales);
  }
  if (a.y == nullptr || n <= 0) return;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    fg[i] = act_of<ACT>(fg[i]);
    if (a.up != nullptr) fg[i] *= fu[i];
  }
  Eight<T, STREAM>::store(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, fg, n);
}

struct ActBackArgs {
  const int8_t* gate_codes;
  const uint8_t* gate_scales;
  const int8_t* up_codes;
  const uint8_t* up_scales;
  const void* dy;
  void* dgate;
  void* dup;
  void* y;
  int64_t ld_dy, ld_dg, ld_du, ld_y;
  uint32_t items, cols, blocks;
  Divider per_row;
};

// Eight kept elements: their codes' bytes, and the scale byte of their block.
struct Kept {
  u32x2_t w;
  uint32_t scale;
  __device__ __forceinline__ void load(const int8_t* codes, const uint8_t* scales, uint32_t row, uint32_t c, int n,
                                       uint32_t cols, uint32_t blocks) {
    w = u32x2_t{0, 0};
    scale = 0;
    if (n <= 0) return;
    const int8_t* p = codes + (int64_t)row * cols + c;
    if (n >= 8) {
      w = *reinterpret_cast<const u32x2_a1*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (i < n) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    }
    scale = scales[(int64_t)row * blocks + c / 32];
  }
  // code * 2^(scale - 133), exact; NaN for a scale of 255.  Codes go from bytes to
  // floats unsigned, 128 above themselves (128 * 2^121 alone would overflow).
  __device__ __forceinline__ void values(float* f) const {
    const float s = scale == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(1.0f, (int)scale - 133);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t b = ((w[i >> 2] ^ 0x80808080u) >> (8 * (i & 3))) & 0xFFu;
      f[i] = ((float)b - 128.0f) * s;
    }
  }
};

template <typename T, int ACT, bool STREAM>
__global__ __launch_bounds__(256) void k_act_back(ActBackArgs a) {
  const uint32_t item = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = divide(item, a.per_row), c = (item - row * a.per_row.d) * 8;
  const int n = item < a.items && c < a.cols ? (int)min(a.cols - c, 8u) : 0;
  if (n <= 0) return;
  Kept kg, ku;
  Eight<T, STREAM> d;
  kg.load(a.gate_codes, a.gate_scales, row, c, n, a.cols, a.blocks);
  if (a.up_codes != nullptr) ku.load(a.up_codes, a.up_scales, row, c, n, a.cols, a.blocks);
  if (a.dy != nullptr) d.load(static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy + c, n);
  float g[8], u[8], dy[8], slope[8];
  kg.values(g);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    u[i] = 1.0f;
    dy[i] = 0.0f;
    g[i] = act_of<ACT, true>(g[i], slope[i]);
  }
  if (a.up_codes != nullptr) ku.values(u);
  if (a.dy != nullptr) d.unpack(dy);
  if (a.dgate != nullptr) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = (dy[i] * u[i]) * slope[i];
    Eight<T, STREAM>::store(static_cast<T*>(a.dgate) + (int64_t)row * a.ld_dg + c, f, n);
  }
  if (a.dup != nullptr) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = dy[i] * g[i];
    Eight<T, STREAM>::store(static_cast<T*>(a.dup) + (int64_t)row * a.ld_du + c, f, n);
  }
  if (a.y != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; i++) g[i] *= u[i];
    Eight<T, STREAM>::store(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, g, n);
  }
}

// Lanes of a row: whole blocks of 32 elements, 8 a lane.
uint32_t lanes_of(int64_t cols) { return (uint32_t)((cols + 31) / 32 * 4); }

}  // namespace

hipError_t launch_gated_act(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                            int64_t ld_g, int64_t ld_u, void* y, int64_t ld_y, int8_t* gate_codes,
                            uint8_t* gate_scales, int8_t* up_codes, uint8_t* up_scales, hipStream_t s) {
  const uint32_t lanes = lanes_of(cols), items = (uint32_t)rows * lanes;
  const ActArgs a{gate, up,   y,    gate_codes, gate_scales,    up_codes,  up_scales,          ld_g,
                  ld_u, ld_y, items, (uint32_t)cols, lanes / 4, make_divider(lanes)};
  const unsigned grid = (items + 255) / 256;
  const int64_t size = dt == 0 ? 2 : 4, tensors = (up == nullptr ? 1 : 2) + (y == nullptr ? 0 : 1);
  const bool stream = rows * cols * tensors * size >= kStreamBytes;
  with_act(act, [&](auto kind) {
    auto* kernel = dt == 0 ? stream ? &k_act<uint16_t, kind.value, true> : &k_act<uint16_t, kind.value, false>
                   : stream ? &k_act<float, kind.value, true>
                            : &k_act<float, kind.value, false>;
    kernel<<<grid, 256, 0, s>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_gated_act_back(int act, const int8_t* gate_codes, const uint8_t* gate_scales, const int8_t* up_codes,
                                 const uint8_t* up_scales, const void* dy, int dt, int64_t rows, int64_t cols,
                                 int64_t ld_dy, void* dgate, int64_t ld_dg, void* dup, int64_t ld_du, void* y,
                                 int64_t ld_y, hipStream_t s) {
  const uint32_t lanes = lanes_of(cols), items = (uint32_t)rows * lanes;
  const ActBackArgs a{gate_codes, gate_scales, up_codes, up_scales, dy,    dgate,          dup,
                      y,          ld_dy,       ld_dg,    ld_du,     ld_y,  items,          (uint32_t)cols,
                      lanes / 4,  make_divider(lanes)};
  const unsigned grid = (items + 255) / 256;
  const int64_t size = dt == 0 ? 2 : 4;
  const int64_t tensors = (dy == nullptr ? 0 : 1) + (dgate == nullptr ? 0 : 1) + (dup == nullptr ? 0 : 1) +
                          (y == nullptr ? 0 : 1);
  const bool stream = rows * cols * tensors * size >= kStreamBytes;
  with_act(act, [&](auto kind) {
    auto* kernel = dt == 0 ? stream ? &k_act_back<uint16_t, kind.value, true> : &k_act_back<uint16_t, kind.value, false>
                   : stream ? &k_act_back<float, kind.value, true>
                            : &k_act_back<float, kind.value, false>;
    kernel<<<grid, 256, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace nvfp4
