/*
 * wino_q8_ops — the operators that stand around the convolutions of
 * wino_q8_conv.h in a UNet: group normalisation with an activation, and the
 * matrix product with bias, activation and residual, forward and backward.
 * Same library, same conventions (wino_q8_conv.h, "Conventions for every entry
 * point"): caller-owned 16-byte aligned device pointers, nothing allocated or
 * synchronised, arguments checked before anything is enqueued, plans immutable
 * and usable from several host threads. Unlike the convolution, both operators
 * define their results for infinities and NaN: they propagate as IEEE
 * arithmetic on the formulas below gives them.
 */
#ifndef WINO_Q8_OPS_H
#define WINO_Q8_OPS_H

#include "wino_q8_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(z). GELU is z Phi(z) with the error function, GELU_TANH its form with
 * tanh(sqrt(2/pi) (z + 0.044715 z^3)). RELU's derivative at 0 is 0. */
typedef enum {
    WQ8_ACT_NONE = 0,
    WQ8_ACT_RELU = 1,
    WQ8_ACT_SILU = 2,
    WQ8_ACT_GELU = 3,
    WQ8_ACT_GELU_TANH = 4
} wq8_act;

/* NHWC: [N][H][W][C], one row of C channels per pixel, rows `stride` elements
 * apart (a slice of a wider tensor is such a one). NCHW: [N][C][H][W],
 * contiguous. */
typedef enum { WQ8_NHWC = 0, WQ8_NCHW = 1 } wq8_layout;

/* ---- Group normalisation with an activation ------------------------------
 * For image n, channel c of group g = c / (C / groups), pixel p, and
 * m = H W C / groups values per (n, g):
 *   v = x + shift[n][c]                      (shift optional: the time
 *                                             embedding a UNet block adds)
 *   mean = sum v / m;  rstd = 1 / sqrt(sum (v - mean)^2 / m + eps)
 *   h = (v - mean) rstd;  z = gamma[c] h + beta[c];  y = act(z)
 * Backward, from dy, x and the forward's mean and rstd:
 *   dz = dy act'(z);  dbeta = sum_{n,p} dz;  dgamma = sum_{n,p} dz h
 *   t = gamma dz;  dx = rstd (t - mean_g t - h mean_g(t h))
 *   dshift[n][c] = sum_p dx
 * All of it in fp32. Squared deviations are summed about the mean, or about
 * the mean of some of a thread's own values with the difference taken off:
 * a mean far from zero costs no more than its own rounding. x and y are
 * rounded to their type once. Sums are taken in a fixed order: results repeat
 * bit for bit. */
typedef struct wq8_norm_plan wq8_norm_plan; /* opaque */

typedef struct {
    int N, C, H, W;          /* N may be 0: an empty batch, nothing is launched but
                                the zeros of dgamma and dbeta. Images of 2^31 values
                                are refused, and those whose last block's pixels or
                                channels would be counted past 2^31 */
    int groups;              /* C % groups == 0 */
    float eps;               /* >= 0, finite */
    wq8_act act;
    wq8_dtype x_dtype;       /* x and dx */
    wq8_dtype y_dtype;       /* y and dy */
    wq8_layout x_layout;     /* x and dx */
    wq8_layout y_layout;     /* y and dy */
    int x_stride, y_stride;  /* NHWC only: elements between pixels, 0 = C */
} wq8_norm_desc;

wq8_status wq8_norm_plan_create(const wq8_norm_desc *desc, wq8_norm_plan **out);
void wq8_norm_plan_destroy(wq8_norm_plan *plan);
/* Workspace bytes of the forward and of the backward (0: none needed, the
 * workspace may be NULL). Either pointer may be NULL. */
wq8_status wq8_norm_plan_query(const wq8_norm_plan *plan, size_t *forward_bytes,
                               size_t *backward_bytes);

/* shift [N][C], gamma [C], beta [C]: f32, each optional (NULL = 0, 1, 0).
 * mean, rstd [N][groups] f32: optional outputs, needed by the backward. x and
 * y must not overlap. */
wq8_status wq8_norm_forward(const wq8_norm_plan *plan, const void *x, const float *shift,
                            const float *gamma, const float *beta, void *y, float *mean,
                            float *rstd, void *workspace, size_t workspace_bytes, void *stream);

/* dgamma, dbeta [C] and dshift [N][C] (f32) are optional outputs; dx is
 * written with x's layout, type and stride. dx must not overlap x or dy. */
wq8_status wq8_norm_backward(const wq8_norm_plan *plan, const void *dy, const void *x,
                             const float *shift, const float *gamma, const float *beta,
                             const float *mean, const float *rstd, void *dx, float *dgamma,
                             float *dbeta, float *dshift, void *workspace, size_t workspace_bytes,
                             void *stream);

/* ---- Matrix product with bias, activation and residual --------------------
 *   z[r][o] = sum_i x[r][i] w[o][i] + bias[o];  y = act(z) + residual
 * r < rows (pixels of all images, or tokens), i < Cin, o < Cout: a 1x1
 * convolution over channels-last activations. Products of bf16 inputs are
 * exact and summed in fp32 on the matrix cores; fp32 inputs use the fp32
 * matrix cores.
 * Backward, from dy and the forward's z (needed unless act is NONE):
 *   dz = dy act'(z);  dx = dz w;  dw = dz^T x;  dbias = sum_r dz
 * and the residual's gradient is dy itself. dz is an fp32 value; with fp32
 * inputs, or where it is a bf16 dy itself, it enters the two products as it
 * is. With bf16 inputs it does so to 16 bits, as the sum of two bf16 values of
 * its sign: dx and dw are then as exact as their own rounding to bf16 leaves
 * them, for twice the matrix work and 4 bytes of workspace a value. A caller
 * who wants it rounded to bf16 once instead (dx and dw off by 2.4e-3 of their
 * norm where 1.7e-3 is their own rounding) asks for it by round_dz. dbias sums
 * fp32 values either way. Sums are taken in a fixed order: results repeat bit
 * for bit. */
typedef struct wq8_linear_plan wq8_linear_plan; /* opaque */

typedef struct {
    int64_t rows;            /* may be 0: nothing is launched but the zeros of dw
                                and dbias */
    int Cin, Cout;
    wq8_act act;
    wq8_dtype x_dtype;       /* x, w, dx and dw */
    wq8_dtype y_dtype;       /* y, z, residual and dy */
    wq8_layout r_layout;     /* residual: NHWC [rows][Cout] (rows r_stride apart), or
                                NCHW [rows / pixels][Cout][pixels], contiguous: what
                                the convolution gives */
    int pixels;              /* pixels per image of an NCHW residual; rows % pixels == 0 */
    int x_stride, y_stride, r_stride; /* elements between rows of x and dx, of y and dy,
                                         and of an NHWC residual; 0 = contiguous */
    int round_dz;            /* backward with bf16 inputs: 0 dz to 16 bits, 1 rounded to
                                bf16; nothing else is changed by it */
} wq8_linear_desc;

wq8_status wq8_linear_plan_create(const wq8_linear_desc *desc, wq8_linear_plan **out);
void wq8_linear_plan_destroy(wq8_linear_plan *plan);
wq8_status wq8_linear_plan_query(const wq8_linear_plan *plan, size_t *forward_bytes,
                                 size_t *backward_bytes);

/* w [Cout][Cin] (x_dtype), bias [Cout] f32 optional, residual (y_dtype)
 * optional, z [rows][Cout] (y_dtype) optional output. y must not overlap x, w,
 * or an NCHW residual; an NHWC residual may be y itself (an addition in
 * place). */
wq8_status wq8_linear_forward(const wq8_linear_plan *plan, const void *x, const void *w,
                              const float *bias, const void *residual, void *y, void *z,
                              void *workspace, size_t workspace_bytes, void *stream);

/* dx, dw [Cout][Cin] (x_dtype) and dbias [Cout] (f32) are optional outputs:
 * what is NULL is not computed. Outputs must not overlap inputs. */
wq8_status wq8_linear_backward(const wq8_linear_plan *plan, const void *dy, const void *x,
                               const void *w, const void *z, void *dx, void *dw, float *dbias,
                               void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WINO_Q8_OPS_H */
