// Declarations shared by the host plans and the kernels of the operators on
// 8-bit codes: packed rows, the root-mean-square norm, the product of codes.
#pragma once

#include "../../include/wino_q8_tokens.h"
#include "wq8_ops_internal.h"

namespace wq8 {

constexpr int code_stride(int columns) { return (columns + 127) / 128 * 128; }

// ------------------------------------------------------- rows held in registers
// A row is held by `lanes` threads, 8 columns of each in `unroll` steps; a block
// has `per` rows. lanes = 0: longer rows, read twice by 1024 threads.
struct RowShape {
    int lanes, unroll, per;
};

struct RowsGeo {
    int rows, C, stride;      // stride: bytes of a row of codes, and the columns that its threads cover
    int64_t xs, ys;
    float eps;
    int group;
    RowShape s;
    int chunk, nchunk;        // norm backward: rows per block, blocks
};

struct RmsPtrs {
    const void *x, *residual, *dy, *dh;
    const float *gamma, *rstd_in;
    void *h, *y, *dx;
    int8_t *codes;
    float *scales, *rstd, *dgamma;
    float *part;              // backward: [nchunk][C]
};

wq8_status launch_rms_forward(const RowsGeo &g, wq8_dtype xdt, wq8_dtype ydt, const RmsPtrs &p, void *stream);
wq8_status launch_rms_backward(const RowsGeo &g, wq8_dtype xdt, wq8_dtype ydt, const RmsPtrs &p, void *stream);
wq8_status launch_pack_rows(const RowsGeo &g, wq8_dtype xdt, const void *x, int8_t *codes, float *scales, void *stream);
wq8_status launch_pack_groups(const RowsGeo &g, wq8_dtype xdt, const void *x, int8_t *codes, float *scales, void *stream);
wq8_status launch_unpack(const RowsGeo &g, wq8_dtype xdt, const int8_t *codes, const float *scales, void *x, void *stream);

// -------------------------------------------------------------- product of codes
// Sums of a block's k steps stay below 2^31: 512 steps of 128 products of
// 128 x 128, and what a lower plane carries.
constexpr int kQ8MaxSteps = 512;

constexpr int kQ8Rows = -1;  // the kernel for up to 2 rows
constexpr int kQ8Thin = -2;  // the kernel for a short batch

struct Q8Shape {
    int tile;      // index into kQ8Tiles (backward: kQ8PairTiles), or one of the below
    int splits, ksteps;
};

struct Q8Geo {
    int M, K, N;              // rows, Cin, Cout
    int Mp, Kp, Np;           // in whole 128-byte lines of codes
    int act;
    int64_t xs, ys, rs;
    int r_planar, pixels;
    int planes;               // 8-bit digits of dz's products: 4, or 2 where the caller asks for them
    Q8Shape f, dx, dw;        // dx and dw share a tile: they run in one kernel
    int chunk, nchunk;        // backward: rows per block of the first pass, blocks along the rows
    int ncol;                 // and along the columns
};

struct Q8Ptrs {
    const int8_t *xq, *wq, *zq_in;
    const float *sx, *sw, *bias, *sz_in;
    const void *residual, *dy, *z_in;
    void *y, *z, *dx, *dw;
    int8_t *zq;
    float *sz, *dbias;
    void *partial, *partial_dx, *partial_dw;  // workspace: split products
    int8_t *xt, *wt;          // workspace: xq [K][Mp] and wq [K][Np] transposed
    int8_t *ur, *uc;          // workspace: digits of dz sw [planes][M][Np] and of dz sx [planes][N][Mp]
    float *rowmax, *colmax, *colsum;  // workspace: [ncol][M], [nchunk][Np], [nchunk][Np]
    float *rscale, *cscale;   // workspace: [M], [N]
};

// Tiles: rows, columns, blocks that a compute unit holds, share of the largest
// tile's rate. The second table is for products of two planes at once.
struct Q8Tile {
    int bm, bn, blocks;
    double rate;
};
constexpr Q8Tile kQ8Tiles[] = {{256, 256, 1, 1.0}, {128, 128, 2, 0.8}, {128, 64, 2, 0.62}, {64, 64, 2, 0.45}};
constexpr Q8Tile kQ8PairTiles[] = {{256, 128, 1, 1.0}, {128, 128, 1, 0.92}, {128, 64, 2, 0.72}, {64, 64, 2, 0.6}};

wq8_status launch_q8_forward(const Q8Geo &g, wq8_dtype ydt, const Q8Ptrs &p, void *stream);
wq8_status launch_q8_backward(const Q8Geo &g, wq8_dtype xdt, wq8_dtype ydt, const Q8Ptrs &p, void *stream);

}  // namespace wq8

struct wq8_quant_plan {
    wq8::RowsGeo geo;
    wq8_dtype xdt;
};

struct wq8_rms_plan {
    wq8::RowsGeo f, b;
    wq8_dtype xdt, ydt;
    size_t f_bytes, b_bytes;
};

struct wq8_q8linear_plan {
    wq8::Q8Geo geo;
    wq8_dtype xdt, ydt;
    size_t f_bytes, b_bytes;
    size_t off_partial_dx, off_partial_dw, off_xt, off_wt, off_ur, off_uc, off_rowmax, off_colmax, off_colsum, off_rscale,
        off_cscale;
};
