/*
 * libnvfp4, the operators of a residual block in eight bits, on gfx950: the
 * product of 8-bit integers with a scale per token and per output channel, and
 * the quantization of its input; the two norms around a block (after it and
 * before the next) with its gate and residual scale, and their backward pass;
 * the gated activation between a block's two products, whose inputs are kept in
 * 8 bits for its backward pass.
 *
 * Status codes, dtype enum, pointer ownership, stream and error conventions:
 * as in nvfp4.h and nvfp4_layers.h: argument errors are found on the host before
 * anything is enqueued, all work is asynchronous on `stream`, every buffer is
 * the caller's, nothing is kept from one call to the next.  Tensors have any
 * column count and any leading dimension ld >= cols (in elements) and need their
 * element's alignment, where nothing else is said; rows * cols < 2^32, with at
 * most 2^28 - 16 rows; zero rows are no error, and sums over them are zero.
 * Arithmetic is FP32 (IEEE binary32), rounded once to the output's type; the logistic
 * function p of v, in activations and gates, is within (5 + 1.25 |v|) 2^-24 of itself, and 0
 * where it is below 2^-126 (SiLU of v < -87.3 is -0).  Infinities and NaN are carried
 * through as IEEE arithmetic carries them, and in 8 bits as said below.  Every result is
 * deterministic.
 *
 * Codes with a scale per row (the product's operands).  amax = the row's largest
 * magnitude; scale = amax / 127; code = nearest even integer of v * (127 / amax),
 * each operation rounded to FP32: codes lie in [-127, 127].  Rows with amax below
 * 2^-100 have scale and codes 0; rows that hold an infinity or a NaN have scale
 * NaN and codes 0.
 *
 * Kept activations.  Blocks of 32 elements along a row (the last of a row may be
 * shorter) share one UE8M0 scale byte, codes are signed 8-bit integers: the value
 * is code * 2^(byte - 133), which is the MX format's INT8 (a code of 64 is 1.0).
 * The byte is the smallest in [0, 254] under which no code exceeds 127; codes
 * are rounded to nearest even and saturate at +-127 (magnitudes above 127 * 2^121 only, the
 * lowest and the largest values of both types among them).  A block that holds an
 * infinity or a NaN has byte 255 and codes 0, and stands for NaN.
 */
#ifndef NVFP4_BLOCKS_H
#define NVFP4_BLOCKS_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(v): v; v * sigmoid(v); v * (1 + tanh(sqrt(2 / pi) * (v + 0.044715 v^3))) / 2; max(v, 0)^2 */
typedef enum { NVFP4_ACT_NONE = 0, NVFP4_ACT_SILU = 1, NVFP4_ACT_GELU = 2, NVFP4_ACT_RELU2 = 3 } nvfp4_act;

/* How a gate tensor becomes the factor: itself, or its logistic function. */
typedef enum { NVFP4_GATE_LINEAR = 0, NVFP4_GATE_SIGMOID = 1 } nvfp4_gate;

/*
 * nvfp4_int8_quantize -- codes and scale of each row of x.
 *   x [rows][ld_x] of type `dt`; codes [rows][ld_codes] int8, 16-byte aligned,
 *   ld_codes a multiple of 16; scales [rows] FP32.  Columns from cols up to the
 *   next multiple of 16 of each row of codes are written as zeros, so that the
 *   rows are operands of a product over that many.  cols >= 1.
 */
nvfp4_status nvfp4_int8_quantize(const void *x, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                                 int8_t *codes, int64_t ld_codes, float *scales, void *stream);

/*
 * nvfp4_int8_quantize_gated -- the same for v = act(gate) * up, unrounded
 * (up NULL: v = act(gate)).  gate [rows][ld_gate], up [rows][ld_up] of type `dt`.
 */
nvfp4_status nvfp4_int8_quantize_gated(int act, const void *gate, const void *up, int dt,
                                       int64_t rows, int64_t cols, int64_t ld_gate, int64_t ld_up,
                                       int8_t *codes, int64_t ld_codes, float *scales, void *stream);

/*
 * nvfp4_int8_gemm -- c[m][n] = (sum_k a[m][k] * b[n][k]) * b_scales[n] * a_scales[m]
 *   with the sum exact (32-bit integers), rounded to FP32 and multiplied by the
 *   scales in this order in FP32; c of type c_dt.
 *   a [M][lda], b [N][ldb] int8 codes (any value), 16-byte aligned, ld multiples of
 *   16 below 2^23 (rows that start on 128-byte lines are read in whole ones, up to a
 *   third sooner); a_scales [M], b_scales [N] FP32; c [M][ldc].  M >= 0, N >= 1,
 *   both < 2^24, M * N <= 2^35; K a multiple of 16 in [16, 131056] (beyond which the sum
 *   could overflow).
 *   workspace: nvfp4_int8_gemm_workspace_size(M, N, K) bytes, 16-byte aligned, in
 *   use until the call's work on `stream` completes; with fewer bytes, or NULL, the
 *   same result takes longer for some shapes.
 */
nvfp4_status nvfp4_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t *a, int64_t lda,
                             const float *a_scales, const int8_t *b, int64_t ldb,
                             const float *b_scales, void *c, int c_dt, int64_t ldc, void *workspace,
                             int64_t workspace_bytes, void *stream);

/* Bytes of workspace nvfp4_int8_gemm uses (host only, no device needed; 0 for many shapes). */
nvfp4_status nvfp4_int8_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t *bytes);

/*
 * nvfp4_block_norms -- what stands between two blocks:
 *   post_rstd = 1 / sqrt(mean_c(x^2) + eps);   o = (x * post_rstd) * post_gamma
 *   h = residual + scale * (g * o);            g = gate, or sigmoid(gate)
 *   pre_rstd = 1 / sqrt(mean_c(h^2) + eps);    y = (h * pre_rstd) * pre_gamma
 * with h unrounded in the last line: the block's output x is normalized, gated,
 * scaled and added to the residual stream, and normalized for the next block.
 *   x [rows][ld_x], residual [rows][ld_r] (or NULL: h = scale * (g * o)), gate
 *   [rows][ld_gate] (or NULL: g = 1; ld_gate 0: one row of gates for all rows),
 *   h [rows][ld_h] (or NULL), y [rows][ld_y] of type `dt`; post_gamma, pre_gamma
 *   [cols] of type gamma_dt; gate_act an nvfp4_gate; post_rstd, pre_rstd [rows]
 *   FP32 (or NULL), which the backward pass takes with x and h.
 *   Exactly one of y and (codes, scales) is given: codes [rows][ld_codes], scales
 *   [rows] hold y as nvfp4_int8_quantize would (of the unrounded y).
 *   h and y may be x or residual (same ld).  cols >= 1, eps >= 0.
 */
nvfp4_status nvfp4_block_norms(const void *x, const void *residual, const void *gate, int dt,
                               int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_r,
                               int64_t ld_gate, int gate_act, const void *post_gamma,
                               const void *pre_gamma, int gamma_dt, float eps, float scale, void *h,
                               int64_t ld_h, void *y, int64_t ld_y, int8_t *codes, int64_t ld_codes,
                               float *scales, float *post_rstd, float *pre_rstd, void *stream);

/*
 * nvfp4_block_norms_backward -- gradient of nvfp4_block_norms at the saved x, h
 * and statistics (y's gradient dy; dh the gradient that reaches h by the residual
 * path, or NULL).  With n = h * pre_rstd, a = dy * pre_gamma, m = x * post_rstd:
 *   t = dh + pre_rstd * (a - n * mean_c(a * n));   dresidual = t
 *   dpre_gamma[c] = sum_r dy * n;   d = scale * t * g;   dpost_gamma[c] = sum_r d * m
 *   b = d * post_gamma;             dx = post_rstd * (b - m * mean_c(b * m))
 *   dgate = scale * t * (m * post_gamma) * g',   g' = 1, or g * (1 - g)
 *   dy, dh, h, x, gate, dx, dresidual [rows][ld] of type `dt`, gate and ld_gate as
 *   above.  dgate is [rows][ld_dgate] of type `dt`, or where ld_gate is 0 the FP32
 *   sum over the rows [cols] (ld_dgate unused).  dpost_gamma, dpre_gamma [cols]
 *   FP32.  Outputs may be NULL, not all of them, dgate is NULL where gate is; an
 *   output may be one of dy, dh, h, x, gate of its own size (same ld).  Sums over rows
 *   run in a fixed order.  Rows narrower than 16 bytes take a workgroup each (2^20 rows of 4
 *   BF16 columns 39 ms, of 8 0.18).
 *   workspace: at least nvfp4_block_norms_backward_workspace_size(rows, cols)
 *   bytes, 4-byte aligned (may be NULL where no sum over rows is asked for, or that
 *   size is 0), in use until the call's work on `stream` completes.  Fewer bytes:
 *   NVFP4_ESHAPE.
 */
nvfp4_status nvfp4_block_norms_backward(const void *dy, const void *dh, const void *h,
                                        const void *x, const void *gate, int dt, int64_t rows,
                                        int64_t cols, int64_t ld_dy, int64_t ld_dh, int64_t ld_h,
                                        int64_t ld_x, int64_t ld_gate, int gate_act,
                                        const void *post_gamma, const void *pre_gamma, int gamma_dt,
                                        const float *post_rstd, const float *pre_rstd, float scale,
                                        void *dx, int64_t ld_dx, void *dresidual, int64_t ld_dr,
                                        void *dgate, int64_t ld_dgate, float *dpost_gamma,
                                        float *dpre_gamma, void *workspace, int64_t workspace_bytes,
                                        void *stream);

/* Bytes of workspace nvfp4_block_norms_backward takes (host only, no device needed). */
nvfp4_status nvfp4_block_norms_backward_workspace_size(int64_t rows, int64_t cols, int64_t *bytes);

/*
 * nvfp4_gated_act -- y = act(gate) * up (up NULL: act(gate)), and its inputs kept
 * in 8 bits for the backward pass.
 *   gate [rows][ld_gate], up [rows][ld_up], y [rows][ld_y] (or NULL) of type `dt`;
 *   gate_codes, up_codes [rows][cols] int8 and gate_scales, up_scales
 *   [rows][ceil(cols / 32)] bytes: the kept gate and up (any alignment).  Codes are
 *   given with their scales, up's only with gate's and with an up, and gate's alone
 *   not where there is an up; y or codes are given.  y (from unrounded inputs) may be
 *   gate or up (same ld).  With NVFP4_ACT_NONE, no up and no y this keeps any tensor.
 */
nvfp4_status nvfp4_gated_act(int act, const void *gate, const void *up, int dt, int64_t rows,
                             int64_t cols, int64_t ld_gate, int64_t ld_up, void *y, int64_t ld_y,
                             int8_t *gate_codes, uint8_t *gate_scales, int8_t *up_codes,
                             uint8_t *up_scales, void *stream);

/*
 * nvfp4_gated_act_backward -- gradient of the above at the kept inputs, with G and
 * U the values that their codes stand for (no up_codes: U = 1):
 *   dgate = dy * U * act'(G);   dup = dy * act(G);   y = act(G) * U
 *   dy, dgate, dup, y [rows][ld] of type `dt`.  dgate, dup and y may be NULL, not
 *   all three; dup needs up_codes; dy is NULL iff dgate and dup are.  dgate, dup or y may
 *   be dy (same ld).  y is the activation formed again (what the next product's weight
 *   gradient takes); with NVFP4_ACT_NONE and no up_codes it restores a kept tensor.
 */
nvfp4_status nvfp4_gated_act_backward(int act, const int8_t *gate_codes, const uint8_t *gate_scales,
                                      const int8_t *up_codes, const uint8_t *up_scales,
                                      const void *dy, int dt, int64_t rows, int64_t cols,
                                      int64_t ld_dy, void *dgate, int64_t ld_dgate, void *dup,
                                      int64_t ld_dup, void *y, int64_t ld_y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_BLOCKS_H */
