// The gated activation y = act(gate) * up whose inputs are kept in 8 bits, and its
// backward pass from them (nvfp4_gated_act, nvfp4_gated_act_backward), for gfx950.
//
// Both are bound by HBM: each element is read and written once, kept inputs one byte
// each and a scale byte per 32 (8192 x 20480 BF16, SiLU: 1.35 GB in 227 us, 5.9 TB/s;
// backward with the activation formed again 1.69 GB in 272, 6.2 TB/s).  A lane takes a
// 16-byte vector of a row, so that a block of 32 is four adjacent lanes (FP32: eight),
// whose largest magnitude takes two or three lane swaps (two vectors a lane took 17.5 us for
// the backward pass of 1025 x 5119 FP32, one 14.4).  A row's blocks are
// counted whole, so lanes past a ragged row's end have nothing to do but take part in those.
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
  uint32_t items, cols, blocks;  // lanes' vectors in all; a row's elements and blocks
  Divider per_row;
};

template <int CTRL>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}

// Codes and scale byte of a lane's vector; every lane of the block takes part.
template <int N>
__device__ __forceinline__ void keep(const float* f, uint32_t row, uint32_t c, int n, uint32_t cols, uint32_t blocks,
                                     int8_t* codes, uint8_t* scales) {
  // the largest magnitude, on the bits: infinities and NaN order above every number
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; i++) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = lane_max<0xB1>(m);  // neighbours, pairs, (FP32) quads
  m = lane_max<0x4E>(m);
  if constexpr (N == 4) m = lane_max<0x141>(m);
  if (n <= 0) return;
  // m = a * 2^E, 1 <= a < 2: 127 = 1.984375 * 2^6, so the exponent is E - 6 for a <=
  // 1.984375 and E - 5 above.  A subnormal's E reads as -127, its limit for -133 is
  // 127 * 2^-133 = 0x7F0000 * 2^-149.  Under the largest exponent, 121, codes saturate on both
  // sides (-128 * 2^121 would be an infinity).
  const bool finite = m < 0x7F800000u;
  int e = (int)(m >> 23) - 127 - 6 + ((m & 0x7FFFFFu) > (m < 0x800000u ? 0x7F0000u : 0x7E0000u) ? 1 : 0);
  e = min(e, 121);
  uint32_t w[N / 4];
#pragma unroll
  for (int u = 0; u < N / 4; u++) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
      t[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(f[4 * u + i], -e), -127.0f, 127.0f) + kToInt;
    w[u] = finite ? bytes_of(t[0], t[1], t[2], t[3]) : 0u;
  }
  int8_t* p = codes + (int64_t)row * cols + c;
  if (n >= N) {
    if constexpr (N == 8)
      *reinterpret_cast<u32x2_a1*>(p) = u32x2_t{w[0], w[1]};
    else
      *reinterpret_cast<u32_a1*>(p) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (i < n) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if ((c & 31) == 0)
    scales[(int64_t)row * blocks + c / 32] = finite ? (uint8_t)(e + 133) : (uint8_t)255;
}

template <typename T, int ACT, bool STREAM>
__global__ __launch_bounds__(256) void k_act(ActArgs a) {
  constexpr int N = VecOf<T>::N;
  const uint32_t item = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = divide(item, a.per_row), c = (item - row * a.per_row.d) * N;
  const int n = item < a.items && c < a.cols ? (int)min(a.cols - c, (uint32_t)N) : 0;
  u32x4_t g = load_row<T, STREAM, false>(static_cast<const T*>(a.gate) + (int64_t)row * a.ld_g, c, n, a.cols);
  u32x4_t u = load_row<T, STREAM, false>(static_cast<const T*>(a.up) + (int64_t)row * a.ld_u, c, a.up == nullptr ? 0 : n,
                                  a.cols);
  end_row<T>(g, n, a.cols);
  end_row<T>(u, n, a.cols);
  float fg[N], fu[N];
  VecOf<T>::unpack(g, fg);
  VecOf<T>::unpack(u, fu);
  if (a.gate_codes != nullptr) {
    keep<N>(fg, row, c, n, a.cols, a.blocks, a.gate_codes, a.gate_scales);
    if (a.up != nullptr) keep<N>(fu, row, c, n, a.cols, a.blocks, a.up_codes, a.up_scales);
  }
  if (a.y == nullptr || n <= 0) return;
#pragma unroll
  for (int i = 0; i < N; i++) {
    fg[i] = act_of<ACT>(fg[i]);
    if (a.up != nullptr) fg[i] *= fu[i];
  }
  store_vec<T, STREAM>(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(fg), n);
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

// N kept elements: their codes' bytes, and the scale byte of their block.
template <int N>
struct Kept {
  uint32_t w[N / 4];
  uint32_t scale;
  __device__ __forceinline__ void load(const int8_t* codes, const uint8_t* scales, uint32_t row, uint32_t c, int n,
                                       uint32_t cols, uint32_t blocks) {
    const int8_t* p = codes + (int64_t)row * cols;
    if (cols >= (uint32_t)N) {  // past the row's end: its last whole vector, shifted
      p += min(c, cols - N);
      uint64_t v;
      if constexpr (N == 8) {
        const u32x2_t u = *reinterpret_cast<const u32x2_a1*>(p);
        v = (uint64_t)u[1] << 32 | u[0];
      } else {
        v = *reinterpret_cast<const u32_a1*>(p);
      }
      v >>= 8 * (N - n);
      w[0] = (uint32_t)v;
      if constexpr (N == 8) w[1] = (uint32_t)(v >> 32);
    } else {
#pragma unroll
      for (int u = 0; u < N / 4; u++) w[u] = 0;
#pragma unroll
      for (int i = 0; i < N; i++)
        if (i < n) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
    }
    scale = scales[(int64_t)row * blocks + c / 32];
  }
  // code * 2^(scale - 133), exact; NaN for a scale of 255.  Codes go from bytes to
  // floats unsigned, 128 above themselves (128 * 2^121 alone would overflow).
  __device__ __forceinline__ void values(float* f) const {
    const float s = scale == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(1.0f, (int)scale - 133);
#pragma unroll
    for (int i = 0; i < N; i++) {
      const uint32_t b = ((w[i >> 2] ^ 0x80808080u) >> (8 * (i & 3))) & 0xFFu;
      f[i] = ((float)b - 128.0f) * s;
    }
  }
};

template <typename T, int ACT, bool STREAM>
__global__ __launch_bounds__(256) void k_act_back(ActBackArgs a) {
  constexpr int N = VecOf<T>::N;
  const uint32_t item = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = divide(item, a.per_row), c = (item - row * a.per_row.d) * N;
  const int n = item < a.items && c < a.cols ? (int)min(a.cols - c, (uint32_t)N) : 0;
  if (n <= 0) return;
  Kept<N> kg, ku;
  kg.load(a.gate_codes, a.gate_scales, row, c, n, a.cols, a.blocks);
  if (a.up_codes != nullptr) ku.load(a.up_codes, a.up_scales, row, c, n, a.cols, a.blocks);
  const u32x4_t d = load_or_zero<T, STREAM>(static_cast<const T*>(a.dy) + (int64_t)row * a.ld_dy, c,
                                            a.dy == nullptr ? 0 : n, a.cols);
  float g[N], u[N], dy[N], slope[N];
  kg.values(g);
  VecOf<T>::unpack(d, dy);
#pragma unroll
  for (int i = 0; i < N; i++) {
    u[i] = 1.0f;
    g[i] = act_of<ACT, true>(g[i], slope[i]);
  }
  if (a.up_codes != nullptr) ku.values(u);
  if (a.dgate != nullptr) {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; i++) f[i] = (dy[i] * u[i]) * slope[i];
    store_vec<T, STREAM>(static_cast<T*>(a.dgate) + (int64_t)row * a.ld_dg + c, VecOf<T>::pack(f), n);
  }
  if (a.dup != nullptr) {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; i++) f[i] = dy[i] * g[i];
    store_vec<T, STREAM>(static_cast<T*>(a.dup) + (int64_t)row * a.ld_du + c, VecOf<T>::pack(f), n);
  }
  if (a.y != nullptr) {
#pragma unroll
    for (int i = 0; i < N; i++) g[i] *= u[i];
    store_vec<T, STREAM>(static_cast<T*>(a.y) + (int64_t)row * a.ld_y + c, VecOf<T>::pack(g), n);
  }
}

// Lanes of a row: whole blocks of 32 elements, 8 or (FP32) 4 a lane.  At most 2^31 in all.
uint32_t lanes_of(int64_t cols, int dt) { return (uint32_t)((cols + 31) / 32 * (dt == 0 ? 4 : 8)); }

}  // namespace

hipError_t launch_gated_act(int act, const void* gate, const void* up, int dt, int64_t rows, int64_t cols,
                            int64_t ld_g, int64_t ld_u, void* y, int64_t ld_y, int8_t* gate_codes,
                            uint8_t* gate_scales, int8_t* up_codes, uint8_t* up_scales, hipStream_t s) {
  const uint32_t lanes = lanes_of(cols, dt), items = (uint32_t)rows * lanes, blocks = (uint32_t)((cols + 31) / 32);
  const ActArgs a{gate, up,   y,    gate_codes, gate_scales,    up_codes,  up_scales,          ld_g,
                  ld_u, ld_y, items, (uint32_t)cols, blocks, make_divider(lanes)};
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
  const uint32_t lanes = lanes_of(cols, dt), items = (uint32_t)rows * lanes, blocks = (uint32_t)((cols + 31) / 32);
  const ActBackArgs a{gate_codes, gate_scales, up_codes, up_scales, dy,    dgate,          dup,
                      y,          ld_dy,       ld_dg,    ld_du,     ld_y,  items,          (uint32_t)cols,
                      blocks,  make_divider(lanes)};
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
