/*
 * libnvfp4, the operators between the quantized layers of a training step and
 * its loss, on gfx950: dropout whose mask is never stored, the residual
 * addition with RMS norm (output in the input's type, or in 8 bits with block
 * scales) and its backward pass, and the softmax cross entropy of a linear
 * head over a large vocabulary, which keeps no logits, with its gradient.
 *
 * Status codes, dtype enum, pointer ownership, stream and error conventions:
 * as in nvfp4.h (argument errors are found on the host before anything is
 * enqueued; all work is asynchronous on `stream`; every buffer, workspaces
 * included, is the caller's; nothing is kept from one call to the next).
 * Differences from nvfp4.h, for all entry points here:
 *   - any column count and any leading dimension ld >= cols (in elements) is
 *     taken, and tensor pointers need only their element's alignment (16 bytes
 *     for the operands of the cross entropy, whose ld are multiples of 8);
 *   - there are at most 2^28 - 16 rows;
 *   - zero rows (tokens) are no error: the call does nothing to per-row outputs
 *     (their pointers may be NULL), and sums over the rows are zero;
 *   - infinities and NaN are carried through as IEEE arithmetic carries them.
 * All arithmetic is in FP32 (IEEE binary32), rounded once to the output's type.
 * Every result is deterministic: it depends only on the arguments.
 *
 * Dropout bits.  Element i = r * cols + c of a rows x cols tensor (the index in
 * the packed tensor, whatever the leading dimension) is kept iff
 * r16(i) >= cut, cut = p * 2^16 rounded to nearest even, with r16 the 16 random
 * bits that nvfp4.h defines for (seed, i).  Kept elements are multiplied by
 * 65536 / (65536 - cut) rounded to FP32; dropped ones are 0 whatever they held.
 * A backward pass repeats the mask from the same seed, rows and cols.
 * 0 <= p < 1 - 2^-17; p = 0 (or cut = 0) keeps everything.
 */
#ifndef NVFP4_LAYERS_H
#define NVFP4_LAYERS_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nvfp4_dropout -- y = dropout(x): also its own backward pass, on the gradient
 * with the forward's seed.
 *   x [rows][ld_x], y [rows][ld_y] of type `dt`; y may be x (same ld).
 *   rows * cols < 2^32.
 */
nvfp4_status nvfp4_dropout(const void *x, int dt, int64_t rows, int64_t cols, int64_t ld_x,
                           float p, uint64_t seed, void *y, int64_t ld_y, void *stream);

/*
 * nvfp4_rms_norm -- residual addition and RMS norm of each row:
 *   h = residual + dropout(x);   rstd = 1 / sqrt(mean_c(h^2) + eps);
 *   y = (h * rstd) * gamma
 * with h unrounded in the second and third.
 *   x [rows][ld_x], residual [rows][ld_r] (or NULL: h = dropout(x)), h
 *   [rows][ld_h] (or NULL), y [rows][ld_y], all of type `dt`; gamma [cols] of
 *   type gamma_dt; rstd [rows] FP32 (or NULL).  h is what the next residual
 *   addition and the backward pass take, rstd what the backward pass takes.
 *   Exactly one of y and (codes, scales) is given.  codes [rows][cols] holds
 *   the norm in 8 bits, scales [rows][ceil(cols / 32)] one UE8M0 exponent byte
 *   per 32 columns (the last block of a row may be shorter): the value is
 *   e4m3(code) * 2^(scale - 127).  The exponent is the smallest under which no
 *   element of the block exceeds 448, in [-127, 127] (-127 for an all-zero
 *   block); codes are rounded to nearest even.  A block that holds an infinity
 *   or a NaN gets scale byte 255 (the format's NaN).
 *   h and y may be x or residual (same ld).  cols >= 1, rows * cols < 2^32,
 *   eps >= 0.
 */
nvfp4_status nvfp4_rms_norm(const void *x, const void *residual, int dt, int64_t rows, int64_t cols,
                            int64_t ld_x, int64_t ld_r, const void *gamma, int gamma_dt, float eps,
                            float p, uint64_t seed, void *h, int64_t ld_h, void *y, int64_t ld_y,
                            uint8_t *codes, uint8_t *scales, float *rstd, void *stream);

/*
 * nvfp4_rms_norm_backward -- gradient of nvfp4_rms_norm at the saved h and rstd
 * (y's gradient dy; dh the gradient that reaches h by the residual path, or
 * NULL).  With n = h * rstd:
 *   g = dh + rstd * (dy * gamma - n * mean_c(dy * gamma * n))
 *   dresidual = g;   dx = dropout(g);   dgamma[c] = sum_r dy[r][c] * n[r][c]
 *   dy, dh, h, dx, dresidual [rows][ld] of type `dt`; dgamma [cols] FP32.  dx,
 *   dresidual and dgamma may each be NULL, not all three; dx and dresidual may
 *   be dy or dh (same ld), not h.  The dgamma sum runs in a fixed order.
 *   workspace: at least nvfp4_rms_norm_backward_workspace_size(rows, cols)
 *   bytes, 4-byte aligned (may be NULL where dgamma is, or where that size is
 *   0), in use until the call's work on `stream` completes.  Fewer bytes:
 *   NVFP4_ESHAPE.
 */
nvfp4_status nvfp4_rms_norm_backward(const void *dy, const void *dh, const void *h, int dt,
                                     int64_t rows, int64_t cols, int64_t ld_dy, int64_t ld_dh,
                                     int64_t ld_h, const void *gamma, int gamma_dt,
                                     const float *rstd, float p, uint64_t seed, void *dx,
                                     int64_t ld_dx, void *dresidual, int64_t ld_dr, float *dgamma,
                                     void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace nvfp4_rms_norm_backward takes (host only, no device needed). */
nvfp4_status nvfp4_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, int64_t *bytes);

/*
 * nvfp4_linear_cross_entropy -- loss of a linear head, token by token:
 *   z[v] = sum_k x[t][k] * w[v][k];  lse[t] = log sum_v exp(z[v]);
 *   loss[t] = lse[t] - z[labels[t]], 0 where labels[t] is outside [0, V)
 * for T tokens, V vocabulary rows and hidden size H.  The logits are formed in
 * tiles and never stored.
 *   x [T][ld_x], w [V][ld_w] BF16, 16-byte aligned, ld a multiple of 8;
 *   labels [T] int64; loss, lse [T] FP32.  H a positive multiple of 8, V >= 1,
 *   T, H and every ld < 2^22, V < 2^24, T * V <= 2^37.
 *   workspace: at least nvfp4_linear_cross_entropy_workspace_size(T, V, H, 0)
 *   bytes, 16-byte aligned, in use until the call's work on `stream` completes.
 *   Fewer bytes: NVFP4_ESHAPE.
 */
nvfp4_status nvfp4_linear_cross_entropy(int64_t T, int64_t V, int64_t H, const void *x,
                                        int64_t ld_x, const void *w, int64_t ld_w,
                                        const int64_t *labels, float *loss, float *lse,
                                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * nvfp4_linear_cross_entropy_backward -- gradient of the above for the loss
 * gradients dloss [T] (FP32), from the forward's lse:
 *   d[t][v] = dloss[t] * (exp(z[t][v] - lse[t]) - (v == labels[t]))
 *   dx[t] = sum_v d[t][v] * w[v];   dw[v] = beta * dw[v] + sum_t d[t][v] * x[t]
 * Tokens whose label is outside [0, V) have d = 0, whatever their x, lse and
 * dloss hold.  The logits are formed again, in pieces of the vocabulary; each
 * d is held as BF16 for the two products, in units of the labelled tokens' largest
 * |dloss| (one rounding, within 2^-8), and with up to 64 labelled tokens in two
 * BF16 parts (within 2^-16).
 *   dx [T][ld_dx] BF16 (or NULL); dw [V][ld_dw] of type dw_dt (or NULL; not
 *   both); 16-byte aligned, ld times element size a multiple of 16.  beta is 0
 *   (overwrite) or 1 (accumulate; the sum is rounded once).  Other arguments as
 *   for the forward; the workspace takes
 *   nvfp4_linear_cross_entropy_workspace_size(T, V, H, 1) bytes and need not
 *   hold anything from the forward.
 */
nvfp4_status nvfp4_linear_cross_entropy_backward(int64_t T, int64_t V, int64_t H, const void *x,
                                                 int64_t ld_x, const void *w, int64_t ld_w,
                                                 const int64_t *labels, const float *lse,
                                                 const float *dloss, void *dx, int64_t ld_dx,
                                                 void *dw, int dw_dt, int64_t ld_dw, float beta,
                                                 void *workspace, int64_t workspace_bytes,
                                                 void *stream);

/* Bytes of workspace for the forward (train 0) or for either direction (train
 * 1) of the linear cross entropy (host only, no device needed). */
nvfp4_status nvfp4_linear_cross_entropy_workspace_size(int64_t T, int64_t V, int64_t H, int train,
                                                       int64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_LAYERS_H */
