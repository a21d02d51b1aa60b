// The linear cross entropy for few tokens (up to 64; the weight gradient up to
// 256), gfx950: every kernel here streams the weight, or its gradient, once past
// the tokens' data and is bound by HBM.
//
// Nothing goes through LDS on the way in: a wave loads its MFMA fragments
// straight into registers, 16 bytes a lane.  MFMA 16 x 16 x 32: lane l = 16 g + i
// holds row i of either operand, k = 8 g .. 8 g + 7; of the result, column i and
// rows 4 g + r, r = 0 .. 3.  Where k runs down a matrix's columns (the rows of W
// in d W, the tokens in d^T x), a lane loads the 8 x 8 block of 8 rows and 8
// adjacent columns, and pairs of rows are interleaved in registers: the j-th of
// the block's columns, taken from all lanes, makes the operand of one matrix
// instruction, whose column i stands for column 8 i + j of the wave's 128.  A
// lane then ends up with 8 adjacent columns of a result row.
#include <algorithm>

#include "layers_launch.hpp"
#include "loss_device.hpp"

namespace nvfp4 {

namespace {

__device__ __forceinline__ bf16x8_t as_frag(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

// Frag j (0 .. C - 1) of the block rows[0..7] (C columns each, C / 2 words): the
// values of column j in row order.
template <int C>
__device__ __forceinline__ bf16x8_t block_column(const uint32_t (&rows)[8][C / 2], int j) {
  const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __builtin_amdgcn_perm(rows[2 * i + 1][j >> 1], rows[2 * i][j >> 1], sel);
  return as_frag(v);
}

// ---- logits of FEW_ROWS vocabulary rows and 16 NT tokens per workgroup
//
// The four waves split the hidden size: wave w takes chunks w, w + 4, .. of 128
// columns, so that together they read 1 KB of each row at a time; their sums meet
// in LDS, in order.
constexpr int CHUNK = 128;

template <int NT>
struct FewChunk {
  u32x4_t a[4][2], b[4][NT];
  __device__ __forceinline__ void load(const uint16_t* const (&wr)[2], const uint16_t* const (&xr)[NT], int c, int H) {
#pragma unroll
    for (int s = 0; s < 4; s++) {
      const int k = c + 32 * s;
#pragma unroll
      for (int q = 0; q < 2; q++) a[s][q] = k < H ? *reinterpret_cast<const u32x4_t*>(wr[q] + k) : u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < NT; q++)
        b[s][q] = k < H ? *reinterpret_cast<const u32x4_t*>(xr[q] + k) : u32x4_t{0, 0, 0, 0};
    }
  }
};

// z[row][token] of the workgroup in LDS (4 waves x 32 rows x 16 NT tokens);
// n >= 1 tokens, rows of the weight from row v0 on.
template <int NT>
__device__ __forceinline__ void few_logits(const uint16_t* w, uint32_t ld_w, int V, int v0, const uint16_t* x,
                                           uint32_t ld_x, int n, int H, float* z) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const uint16_t* wr[2];
  const uint16_t* xr[NT];
#pragma unroll
  for (int q = 0; q < 2; q++) wr[q] = w + (int64_t)min(v0 + 16 * q + i, V - 1) * ld_w;
#pragma unroll
  for (int q = 0; q < NT; q++) xr[q] = x + (int64_t)min(16 * q + i, n - 1) * ld_x;
  floatx4 acc[2][NT];
#pragma unroll
  for (int q = 0; q < 2; q++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[q][t] = floatx4{0, 0, 0, 0};
  FewChunk<NT> cur, nxt;
  const int c0 = wave * CHUNK + 8 * g;  // the lane's first column; H is a multiple of 8
  cur.load(wr, xr, c0, H);
  for (int c = wave * CHUNK; c < H; c += 4 * CHUNK) {
    nxt.load(wr, xr, c + 4 * CHUNK + 8 * g, H);
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
      for (int q = 0; q < 2; q++)
#pragma unroll
        for (int t = 0; t < NT; t++)
          acc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(cur.a[s][q]), as_frag(cur.b[s][t]), acc[q][t], 0,
                                                              0, 0);
    cur = nxt;
  }
#pragma unroll
  for (int q = 0; q < 2; q++)
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int r = 0; r < 4; r++)
        z[(wave * FEW_ROWS + 16 * q + 4 * g + r) * (16 * NT) + 16 * t + i] = acc[q][t][r];
  __syncthreads();
}

// Thread's token and its first of R consecutive rows: 256 / (16 NT) threads a token.
template <int NT>
struct FewPlace {
  static constexpr int PER = 16 / NT, R = FEW_ROWS / PER;
  int t, row;
  __device__ __forceinline__ FewPlace() : t(threadIdx.x / PER), row(threadIdx.x % PER * R) {}
  __device__ __forceinline__ float logit(const float* z, int r) const {
    float v = z[(row + r) * (16 * NT) + t];
#pragma unroll
    for (int w = 1; w < 4; w++) v += z[(w * FEW_ROWS + row + r) * (16 * NT) + t];
    return v;
  }
};

template <int NT>
__global__ __launch_bounds__(256) void k_few_stats(const uint16_t* w, uint32_t ld_w, int V, const uint16_t* x,
                                                   uint32_t ld_x, int T, int H, const int64_t* labels, float2* stats,
                                                   float* zlab) {
  __shared__ float z[4 * FEW_ROWS * 16 * NT];
  const int v0 = blockIdx.x * FEW_ROWS;
  few_logits<NT>(w, ld_w, V, v0, x, ld_x, T, H, z);
  const FewPlace<NT> p;
  constexpr int R = FewPlace<NT>::R;
  float v[R], mx = -INFINITY;
#pragma unroll
  for (int r = 0; r < R; r++) {
    v[r] = v0 + p.row + r < V ? p.logit(z, r) : -INFINITY;
    mx = fmaxf(mx, v[r]);
  }
  if (p.t < T) {
    const int64_t label = labels[p.t];
    const int lab = label >= 0 && label < V ? (int)label - v0 - p.row : -1;
#pragma unroll
    for (int r = 0; r < R; r++)
      if (lab == r) zlab[p.t] = v[r];
  }
#pragma unroll
  for (int m = 1; m < FewPlace<NT>::PER; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m, 64));
  const float sh = shift_of(mx);
  float s = 0.0f;
#pragma unroll
  for (int r = 0; r < R; r++) s += exp_fast(v[r] - sh);
#pragma unroll
  for (int m = 1; m < FewPlace<NT>::PER; m <<= 1) s += __shfl_xor(s, m, 64);
  if (p.t < T && p.row == 0) stats[(int64_t)p.t * gridDim.x + blockIdx.x] = make_float2(mx, s);
}

template <int NT>
__global__ __launch_bounds__(256) void k_few_grad(const uint16_t* w, uint32_t ld_w, int V, const uint16_t* xc, int H,
                                                  Tokens tk, const int64_t* labels, const float* lse,
                                                  const float* dloss, uint16_t* dt, int ldt, uint16_t* d) {
  __shared__ float z[4 * FEW_ROWS * 16 * NT];
  const int n = *tk.n;
  const int v0 = blockIdx.x * FEW_ROWS;
  const int64_t ldd = (int64_t)gridDim.x * FEW_ROWS;
  if (n > 0) few_logits<NT>(w, ld_w, V, v0, xc, (uint32_t)H, n, H, z);
  const FewPlace<NT> p;
  constexpr int R = FewPlace<NT>::R;
  float v[R];
#pragma unroll
  for (int r = 0; r < R; r++) v[r] = 0.0f;
  if (p.t < n) {
    const int t = tk.list[p.t];
    const float l = lse[t], g = dloss[t];
    const int lab = (int)(labels[t] - v0) - p.row;  // a label lies in [0, V), V < 2^24
#pragma unroll
    for (int r = 0; r < R; r++)
      if (v0 + p.row + r < V) v[r] = g * (exp_fast(p.logit(z, r) - l) - (lab == r ? 1.0f : 0.0f));
  }
  uint32_t* dr = reinterpret_cast<uint32_t*>(d + p.t * ldd + v0 + p.row);
#pragma unroll
  for (int r = 0; r < R; r += 2) {
    const uint32_t q = bf16_pack(v[r], v[r + 1]);
    dr[r / 2] = q;
    dt[(int64_t)(v0 + p.row + r) * ldt + p.t] = (uint16_t)q;
    dt[(int64_t)(v0 + p.row + r + 1) * ldt + p.t] = (uint16_t)(q >> 16);
  }
  if constexpr (NT == 1) {  // columns 16 .. 31 of d^T are K of the dw product
    for (int e = threadIdx.x; e < FEW_ROWS * 8; e += 256)
      reinterpret_cast<uint32_t*>(dt + (int64_t)(v0 + e / 8) * ldt + 16)[e % 8] = 0;
  }
}

// ---- sum[part][t][h] = sum over the part's vocabulary rows of d[t][v] w[v][h]
//
// A workgroup takes 128 columns and a range of steps of 32 rows; its waves take
// the steps in turn, and their sums meet in LDS, in order.
struct WBlock {
  uint32_t r[8][4];
};

template <int NT>
__global__ __launch_bounds__(256) void k_few_dx(const uint16_t* w, uint32_t ld_w, int V, const uint16_t* d, int64_t ldd,
                                                int H, int slices, int parts, Tokens tk, int T, float* sum) {
  __shared__ float red[16 * NT * 128];
  const int n = *tk.n;
  if (n == 0) return;
  const int slice = blockIdx.x % slices, part = blockIdx.x / slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int steps = (V + 31) / 32;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  const int h = slice * 128 + 8 * i;
  const uint16_t* wc = w + min(h, H - 8);
  const uint16_t* dr = d + (int64_t)i * ldd + 8 * g;
  floatx4 acc[NT][8];
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int j = 0; j < 8; j++) acc[t][j] = floatx4{0, 0, 0, 0};
  auto load = [&](int s, WBlock& b, u32x4_t (&a)[NT]) {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      // rows past V: their d is 0
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(wc + (int64_t)min(32 * s + 8 * g + j, V - 1) * ld_w);
#pragma unroll
      for (int q = 0; q < 4; q++) b.r[j][q] = v[q];
    }
#pragma unroll
    for (int t = 0; t < NT; t++) a[t] = *reinterpret_cast<const u32x4_t*>(dr + 16 * t * ldd + 32 * s);
  };
  WBlock cur, nxt;
  u32x4_t ca[NT], na[NT];
  if (s0 + wave < s1) load(s0 + wave, cur, ca);
  for (int s = s0 + wave; s < s1; s += 4) {
    load(min(s + 4, s1 - 1), nxt, na);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const bf16x8_t b = block_column<8>(cur.r, j);
#pragma unroll
      for (int t = 0; t < NT; t++)
        acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(ca[t]), b, acc[t][j], 0, 0, 0);
    }
    cur = nxt;
#pragma unroll
    for (int t = 0; t < NT; t++) ca[t] = na[t];
  }
#pragma unroll 1
  for (int q = 3; q > 0; q--) {  // waves 3, 2, 1 hand theirs to the one before
    __syncthreads();
    if (wave == q) {
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) red[((t * 8 + j) * 4 + r) * 64 + lane] = acc[t][j][r];
    }
    __syncthreads();
    if (wave == q - 1) {
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[t][j][r] += red[((t * 8 + j) * 4 + r) * 64 + lane];
    }
  }
  if (wave != 0 || h >= H) return;
#pragma unroll
  for (int t = 0; t < NT; t++)
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int tok = 16 * t + 4 * g + r;
      if (tok >= n) continue;
      float4* o = reinterpret_cast<float4*>(sum + ((int64_t)part * T + tok) * H + h);
      o[0] = make_float4(acc[t][0][r], acc[t][1][r], acc[t][2][r], acc[t][3][r]);
      o[1] = make_float4(acc[t][4][r], acc[t][5][r], acc[t][6][r], acc[t][7][r]);
    }
}

// ---- dw[v][h] (+)= sum_t dt[v][t] xc[t][h]
//
// A wave holds 32 KT tokens of C columns per lane (16 C columns in all) of xc in
// registers and walks the vocabulary 16 rows at a time; the four waves take
// adjacent columns of the same rows.
template <int KT, int C, typename OutT>
__global__ __launch_bounds__(256) void k_few_dw(const uint16_t* xc, int H, const uint16_t* dt, int64_t ldt, int rows,
                                                int slices, int parts, Tokens tk, OutT* dw, int64_t ld_dw,
                                                int accumulate) {
  const int kt = (*tk.n + 31) / 32;  // blocks of 32 tokens that hold any
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
    for (int j = 0; j < C; j++) xf[k][j] = block_column<C>(r, j);
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
      for (int j = 0; j < C; j++) f[j] = acc[j][r];
      if constexpr (sizeof(OutT) == 4) {
#pragma unroll
        for (int j = 0; j < C; j += 4) {
          float4* p = reinterpret_cast<float4*>(o + j);
          float4 s = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
          if (accumulate) {
            const float4 old = *p;
            s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
          }
          *p = s;
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
        if constexpr (C == 8)
          *reinterpret_cast<u32x4_t*>(p) = u32x4_t{b[0], b[1], b[2], b[3]};
        else
          *reinterpret_cast<u32x2_t*>(p) = u32x2_t{b[0], b[1]};
      }
    }
#pragma unroll
    for (int k = 0; k < KT; k++) cur[k] = nxt[k];
  }
}

template <typename F>
hipError_t by_tokens(int64_t T, F&& f) {
  if (T <= 16)
    f(std::integral_constant<int, 1>{});
  else if (T <= 32)
    f(std::integral_constant<int, 2>{});
  else
    f(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

// Workgroups that keep a 256-CU MI355X streaming.
constexpr int64_t kStreams = 1024;

}  // namespace

hipError_t few_stats(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* x, uint32_t ld_x, int64_t T,
                     int64_t H, const int64_t* labels, float2* stats, float* zlab, hipStream_t s) {
  return by_tokens(T, [&](auto nt) {
    k_few_stats<nt.value><<<(unsigned)(few_rows(V) / FEW_ROWS), 256, 0, s>>>(w, ld_w, (int)V, x, ld_x, (int)T, (int)H,
                                                                            labels, stats, zlab);
  });
}

hipError_t few_grad(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* xc, int64_t T, int64_t H, Tokens tk,
                    const int64_t* labels, const float* lse, const float* dloss, uint16_t* dt, uint16_t* d,
                    hipStream_t s) {
  return by_tokens(T, [&](auto nt) {
    k_few_grad<nt.value><<<(unsigned)(few_rows(V) / FEW_ROWS), 256, 0, s>>>(w, ld_w, (int)V, xc, (int)H, tk, labels,
                                                                           lse, dloss, dt, (int)few_ldt(T), d);
  });
}

// Enough workgroups to stream, each of its waves with four steps or more.
int64_t few_dx_parts(int64_t T, int64_t V, int64_t H) {
  const int64_t slices = (H + 127) / 128, steps = (V + 31) / 32;
  const int64_t want = (kStreams / (few_tokens(T) / 16 > 2 ? 2 : 1) + slices - 1) / slices;
  return std::max<int64_t>(1, std::min(want, steps / 16));
}

hipError_t few_dx(const uint16_t* w, uint32_t ld_w, int64_t V, const uint16_t* d, int64_t T, int64_t H, Tokens tk,
                  float* sum, hipStream_t s) {
  const int64_t slices = (H + 127) / 128, parts = few_dx_parts(T, V, H);
  return by_tokens(T, [&](auto nt) {
    k_few_dx<nt.value><<<(unsigned)(slices * parts), 256, 0, s>>>(w, ld_w, (int)V, d, few_rows(V), (int)H, (int)slices,
                                                                  (int)parts, tk, (int)T, sum);
  });
}

template <typename OutT>
static hipError_t few_dw_t(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T,
                           Tokens tk, OutT* dw, int64_t ld_dw, int accumulate, hipStream_t s) {
  auto go = [&](auto kt, auto c) {
    const int64_t slices = (H + 64 * c.value - 1) / (64 * c.value), groups = (rows + 15) / 16;
    const int64_t parts = std::max<int64_t>(1, std::min((2 * kStreams + slices - 1) / slices, groups / 4));
    k_few_dw<kt.value, c.value><<<(unsigned)(slices * parts), 256, 0, s>>>(
        xc, (int)H, dt, ldt, (int)rows, (int)slices, (int)parts, tk, dw, ld_dw, accumulate);
  };
  using std::integral_constant;
  if (T <= 32)
    go(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  else if (T <= 64)
    go(integral_constant<int, 2>{}, integral_constant<int, 8>{});
  else if (T <= 128)
    go(integral_constant<int, 4>{}, integral_constant<int, 8>{});
  else
    go(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t few_dw(const uint16_t* xc, int64_t H, const uint16_t* dt, int64_t ldt, int64_t rows, int64_t T, Tokens tk,
                  void* dw, int dw_f32, int64_t ld_dw, int accumulate, hipStream_t s) {
  if (dw_f32) return few_dw_t(xc, H, dt, ldt, rows, T, tk, static_cast<float*>(dw), ld_dw, accumulate, s);
  return few_dw_t(xc, H, dt, ldt, rows, T, tk, static_cast<uint16_t*>(dw), ld_dw, accumulate, s);
}

}  // namespace nvfp4
