// The weight gradient of the linear cross entropy for few tokens, gfx950:
// dw = d^T x is bound by writing dw to HBM, so the tokens' data stays in registers
// and the kernel streams past it.
//
// A wave loads its MFMA fragments straight into registers, 16 bytes a lane.  MFMA
// 16 x 16 x 32: lane l = 16 g + i holds row i of either operand, k = 8 g .. 8 g + 7;
// of the result, column i and rows 4 g + r, r = 0 .. 3.  k runs down the columns of
// x: a lane loads the 8 x 8 block of 8 tokens and 8 adjacent columns, and pairs of
// rows are interleaved in registers: the j-th of the block's columns, taken from
// all lanes, makes the operand of one matrix instruction, whose column i stands for
// column 8 i + j of the wave's 128.  A lane then ends up with 8 adjacent columns of
// a row of dw, one 16-byte store.
// 131072 x 5120 BF16: 0.28 ms at 16 tokens in two parts (4.8 TB/s; a plain store loop
// reaches 5.3).  From 33 tokens on the tiles are level or better (47 x 16555 x 2264
// 64 us in all against 53).
#include <algorithm>

#include "layers_launch.hpp"
#include "loss_device.hpp"

namespace nvfp4 {

namespace {

__device__ __forceinline__ bf16x8_t as_frag(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

constexpr int C = 8;  // columns a lane holds

// Fragment j of the block rows[0 .. 7]: the values of column j in row order.
__device__ __forceinline__ bf16x8_t block_column(const uint32_t (&rows)[8][C / 2], int j) {
  const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __builtin_amdgcn_perm(rows[2 * i + 1][j >> 1], rows[2 * i][j >> 1], sel);
  return as_frag(v);
}

// ---- dw[v][h] (+)= sum_t dt[v][t] xc[t][h]
//
// A wave holds 32 KT rows (tokens, in two parts) of C columns per lane (128 columns in all) of xc in
// registers and walks the vocabulary 16 rows at a time; the four waves take
// adjacent columns of the same rows.
template <int KT, bool STREAM, typename OutT>
__global__ __launch_bounds__(256) void k_few_dw(const uint16_t* xc, int H, const uint16_t* dt, int64_t ldt, int rows,
                                                int slices, int parts, Tokens tk, OutT* dw, int64_t ld_dw,
                                                int accumulate) {
  const float scale = *tk.scale;
  const int kt = (tk.columns() + 31) / 32;  // blocks of 32 columns that hold any
  const int slice = blockIdx.x % slices, part = blockIdx.x / slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int h = (slice * 4 + wave) * 16 * C + C * i;
  const int hc = min(h, H - C);  // H is a multiple of 8
  bf16x8_t xf[KT][C];
#pragma unroll
  for (int k = 0; k < KT; k++) {
    uint32_t r[8][C / 2];
#pragma unroll
    for (int j = 0; j < 8; j++) {
#pragma unroll
      for (int q = 0; q < C / 2; q++) r[j][q] = 0;
      if (k < kt) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(xc + (int64_t)(32 * k + 8 * g + j) * H + hc);
#pragma unroll
        for (int q = 0; q < C / 2; q++) r[j][q] = p[q];
      }
    }
#pragma unroll
    for (int j = 0; j < C; j++) xf[k][j] = block_column(r, j);
  }
  const int groups = (rows + 15) / 16;
  const int g0 = (int)((int64_t)groups * part / parts), g1 = (int)((int64_t)groups * (part + 1) / parts);
  auto load = [&](int q, u32x4_t (&a)[KT]) {
    const uint16_t* p = dt + (int64_t)min(16 * q + i, rows - 1) * ldt + 8 * g;
#pragma unroll
    for (int k = 0; k < KT; k++)
      if (k < kt) a[k] = *reinterpret_cast<const u32x4_t*>(p + 32 * k);
  };
  u32x4_t cur[KT], nxt[KT];
#pragma unroll
  for (int k = 0; k < KT; k++) cur[k] = nxt[k] = u32x4_t{0, 0, 0, 0};
  if (g0 < g1) load(g0, cur);
#pragma unroll 2
  for (int q = g0; q < g1; q++) {
    load(min(q + 1, g1 - 1), nxt);
    floatx4 acc[C];
#pragma unroll
    for (int j = 0; j < C; j++) acc[j] = floatx4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KT; k++)
      if (k < kt) {
#pragma unroll
        for (int j = 0; j < C; j++)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(cur[k]), xf[k][j], acc[j], 0, 0, 0);
      }
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int v = 16 * q + 4 * g + r;
      if (v >= rows || h >= H) continue;
      OutT* o = dw + (int64_t)v * ld_dw + h;
      float f[C];
#pragma unroll
      for (int j = 0; j < C; j++) f[j] = acc[j][r] * scale;
      if constexpr (sizeof(OutT) == 4) {
#pragma unroll
        for (int j = 0; j < C; j += 4) {
          float4* p = reinterpret_cast<float4*>(o + j);
          float4 s = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
          if (accumulate) {
            const float4 old = *p;
            s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
          }
          store16<STREAM>(p, __builtin_bit_cast(u32x4_t, s));
        }
      } else {
        uint32_t* p = reinterpret_cast<uint32_t*>(o);
        uint32_t b[C / 2];
        if (accumulate) {
#pragma unroll
          for (int j = 0; j < C / 2; j++) {
            f[2 * j] += bf16lo(p[j]);
            f[2 * j + 1] += bf16hi(p[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < C / 2; j++) b[j] = bf16_pack(f[2 * j], f[2 * j + 1]);
        store16<STREAM>(p, u32x4_t{b[0], b[1], b[2], b[3]});
      }
    }
#pragma unroll
    for (int k = 0; k < KT; k++) cur[k] = nxt[k];
  }
}

// Workgroups that keep a 256-CU MI355X streaming.
constexpr int64_t kStreams = 1024;

}  // namespace

template <typename OutT>
static hipError_t few_dw_t(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T,
                           Tokens tk, OutT* dw, int64_t ld_dw, int accumulate, bool stream, hipStream_t s) {
  auto go = [&](auto kt) {
    const int64_t slices = (H + 64 * C - 1) / (64 * C), groups = (rows + 15) / 16;
    const int64_t parts = std::max<int64_t>(1, std::min((2 * kStreams + slices - 1) / slices, groups / 4));
    auto* kernel = stream ? &k_few_dw<kt.value, true, OutT> : &k_few_dw<kt.value, false, OutT>;
    kernel<<<(unsigned)(slices * parts), 256, 0, s>>>(xc, (int)H, dt, ldt, (int)rows, (int)slices, (int)parts, tk, dw,
                                                      ld_dw, accumulate);
  };
  using std::integral_constant;
  if (T <= 16)
    go(integral_constant<int, 1>{});
  else
    go(integral_constant<int, 2>{});
  return hipGetLastError();
}

hipError_t few_dw(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T, Tokens tk,
                  void* dw, int dw_f32, int64_t ld_dw, int accumulate, bool stream, hipStream_t s) {
  if (dw_f32) return few_dw_t(xc, H, dt, ldt, rows, T, tk, static_cast<float*>(dw), ld_dw, accumulate, stream, s);
  return few_dw_t(xc, H, dt, ldt, rows, T, tk, static_cast<uint16_t*>(dw), ld_dw, accumulate, stream, s);
}

}  // namespace nvfp4
