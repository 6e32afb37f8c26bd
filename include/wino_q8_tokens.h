/*
 * wino_q8_tokens — operators of a transformer block's products in 8 bits:
 * packing of rows to codes with scales, the root-mean-square norm with the
 * residual's addition and an output in codes, and the matrix product of codes
 * with scales for each token and channel, with its backward from what was kept
 * in codes. Same library, same conventions as wino_q8_ops.h: caller-owned
 * 16-byte aligned device pointers, nothing allocated or synchronised,
 * arguments checked before anything is enqueued, plans immutable and usable
 * from several host threads, sums in a fixed order: results repeat bit for bit.
 *
 * Codes. `a` being the largest magnitude of a row, or of a group of columns of
 * a row, its values x are held as
 *   code = rint(x (127 / a)), int8 in [-127, 127];  scale = a / 127 (f32)
 * and stand for code * scale. Quotients and products are rounded to f32 each;
 * rint takes ties to even. a = 0: codes and scale 0. Where 127 / a would
 * overflow, x and a are taken times 2^64. An infinity or a NaN anywhere in the
 * row or group: its codes are 0 and its scale NaN, so that it stands for NaN.
 * A row of codes takes whole 128-byte lines (WQ8_CODE_STRIDE bytes): products
 * read lines. Those behind the last column are zero.
 */
#ifndef WINO_Q8_TOKENS_H
#define WINO_Q8_TOKENS_H

#include "wino_q8_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WQ8_CODE_STRIDE(columns) (((columns) + 127) / 128 * 128)

/* ---- Rows to codes and back ------------------------------------------------
 * Activations of a product (group 0: one scale a row), its weights (one scale an
 * output channel), and tensors kept in 8 bits for a backward pass. */
typedef struct wq8_quant_plan wq8_quant_plan; /* opaque */

typedef struct {
    int64_t rows;            /* may be 0: nothing is launched */
    int C;                   /* columns, below 2^20 */
    int group;               /* columns that share a scale: 0 (all), 32, 64 or 128 */
    wq8_dtype x_dtype;
    int x_stride;            /* elements between rows of x, 0 = C */
} wq8_quant_desc;

wq8_status wq8_quant_plan_create(const wq8_quant_desc *desc, wq8_quant_plan **out);
void wq8_quant_plan_destroy(wq8_quant_plan *plan);

/* codes [rows][WQ8_CODE_STRIDE(C)]; scales [rows][groups], groups = 1 (group 0)
 * or ceil(C / group). */
wq8_status wq8_quant_pack(const wq8_quant_plan *plan, const void *x, int8_t *codes, float *scales,
                          void *stream);
/* x = code * scale, rounded to its type. */
wq8_status wq8_quant_unpack(const wq8_quant_plan *plan, const int8_t *codes, const float *scales,
                            void *x, void *stream);

/* ---- Root-mean-square norm with the residual's addition -------------------
 *   h = x + residual, rounded to x's type (the stream; without residual x)
 *   rstd = 1 / sqrt(sum_c h^2 / C + eps);  y = (h rstd) gamma
 * and in codes: those of h gamma, whose scales are taken times rstd (the factor
 * is one for the whole row, so the codes do not depend on it).
 * Backward, from dy, h and rstd; dh is what reaches the stream on its own way:
 *   n = h rstd;  t = gamma dy;  dx = rstd (t - n sum_c(t n) / C) + dh
 *   dgamma = sum_r dy n
 * dx is the gradient of x and of the residual. All of it in fp32. */
typedef struct wq8_rms_plan wq8_rms_plan; /* opaque */

typedef struct {
    int64_t rows;            /* may be 0: nothing is launched but the zeros of dgamma */
    int C;                   /* below 2^20 */
    float eps;               /* >= 0, finite */
    wq8_dtype x_dtype;       /* x, residual, h, dh and dx */
    wq8_dtype y_dtype;       /* y and dy */
    int x_stride, y_stride;  /* elements between rows of x, residual, h, dh and dx, and of y
                                and dy; 0 = C */
} wq8_rms_desc;

wq8_status wq8_rms_plan_create(const wq8_rms_desc *desc, wq8_rms_plan **out);
void wq8_rms_plan_destroy(wq8_rms_plan *plan);
wq8_status wq8_rms_plan_query(const wq8_rms_plan *plan, size_t *forward_bytes,
                              size_t *backward_bytes);

/* gamma [C] f32 optional (NULL = 1). residual optional; with it h may be
 * written, which may be x or residual itself. y, or codes [rows][WQ8_CODE_STRIDE(C)]
 * with scales [rows], or all three. rstd [rows] optional, needed by the
 * backward. y must not overlap another buffer. */
wq8_status wq8_rms_forward(const wq8_rms_plan *plan, const void *x, const void *residual,
                           const float *gamma, void *h, void *y, int8_t *codes, float *scales,
                           float *rstd, void *workspace, size_t workspace_bytes, void *stream);

/* dh optional, and may be dx itself. dgamma [C] optional. dx must not overlap
 * dy or h. */
wq8_status wq8_rms_backward(const wq8_rms_plan *plan, const void *dy, const void *h,
                            const float *rstd, const float *gamma, const void *dh, void *dx,
                            float *dgamma, void *workspace, size_t workspace_bytes, void *stream);

/* ---- Matrix product of codes ----------------------------------------------
 *   z[r][o] = (sum_i xq[r][i] wq[o][i]) sx[r] sw[o] + bias[o]
 *   y = act(z) + residual
 * xq and wq are rows of codes with one scale each (group 0 above). The sums are
 * exact whole numbers; what follows is in fp32. z may be kept for the backward
 * as it is (y_dtype) or in codes with a scale for every 32 columns.
 * Backward, from dy, z and the forward's codes: with dz = dy act'(z), x^ = sx xq
 * and w^ = sw wq, what the codes stand for,
 *   dx = dz w^;  dw = dz^T x^;  dbias = sum_r dz
 * so no 16- or 32-bit activation or weight is read. dz sw (for dx) and dz sx (for
 * dw) are multiplied as whole numbers in fixed point of the largest magnitude m of
 * their row (column), which is 127 256^3 units: each is off by at most half a unit,
 * m / 4261412864, and by its own rounding to f32. With round_dz, where dx and dw are
 * bf16, m is 127 256 units and half a unit m / 65024; where a row (column) holds one
 * value some hundred times the others, that is more than bf16 results lose by
 * themselves. Sums of products are whole numbers: those of round_dz exact, the others
 * to 2^-17 m / 127 (in units of the codes). A sum that is split over several blocks
 * is joined from parts in f32, each with its rounding, in a fixed order. dbias
 * sums fp32 values. A row of dz sw that holds an infinity or a NaN makes its row
 * of dx NaN, a column of dz sx its row of dw. */
typedef struct wq8_q8linear_plan wq8_q8linear_plan; /* opaque */

#define WQ8_Z_GROUP 32

typedef struct {
    int64_t rows;            /* may be 0: nothing is launched but the zeros of dw and dbias */
    int Cin, Cout;           /* below 2^20 */
    wq8_act act;
    wq8_dtype x_dtype;       /* dx and dw */
    wq8_dtype y_dtype;       /* y, z, residual and dy */
    wq8_layout r_layout;     /* residual: as wq8_linear_desc has it */
    int pixels;
    int x_stride, y_stride, r_stride; /* elements between rows of dx, of y and dy, and of an
                                         NHWC residual; 0 = contiguous */
    int round_dz;            /* backward to bf16: dz in 16 bits, for half the matrix work */
} wq8_q8linear_desc;

wq8_status wq8_q8linear_plan_create(const wq8_q8linear_desc *desc, wq8_q8linear_plan **out);
void wq8_q8linear_plan_destroy(wq8_q8linear_plan *plan);
wq8_status wq8_q8linear_plan_query(const wq8_q8linear_plan *plan, size_t *forward_bytes,
                                   size_t *backward_bytes);

/* xq [rows][WQ8_CODE_STRIDE(Cin)], sx [rows], wq [Cout][WQ8_CODE_STRIDE(Cin)],
 * sw [Cout], bias [Cout] f32 optional, residual optional. Outputs beside y, all
 * optional: z [rows][Cout]; zq [rows][WQ8_CODE_STRIDE(Cout)] with sz
 * [rows][ceil(Cout / 32)]. Codes behind the last column of zq are zero.
 * Outputs must not overlap inputs or each other, except that an NHWC residual may
 * be y itself (with y's row stride). */
wq8_status wq8_q8linear_forward(const wq8_q8linear_plan *plan, const int8_t *xq, const float *sx,
                                const int8_t *wq, const float *sw, const float *bias,
                                const void *residual, void *y, void *z, int8_t *zq, float *sz,
                                void *workspace, size_t workspace_bytes, void *stream);

/* Unless act is NONE: z, or zq with sz, one of the two. dx, dw [Cout][Cin]
 * (x_dtype) and dbias [Cout] (f32) are optional outputs: what is NULL is not
 * computed. Outputs must not overlap inputs. */
wq8_status wq8_q8linear_backward(const wq8_q8linear_plan *plan, const void *dy, const int8_t *xq,
                                 const float *sx, const int8_t *wq, const float *sw, const void *z,
                                 const int8_t *zq, const float *sz, void *dx, void *dw,
                                 float *dbias, void *workspace, size_t workspace_bytes,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WINO_Q8_TOKENS_H */
