// Declarations shared by the host plans and the kernels of the group norm and
// the matrix product.
#pragma once

#include "../../include/wino_q8_ops.h"
#include "wq8_internal.h"

namespace wq8 {

// Compute units of an MI355X: launch shapes are chosen when a plan is made,
// where no device need be present.
constexpr int kCus = 256;

// ------------------------------------------------------------- group norm
constexpr int kNormMaxSlab = 1024;  // channels per block

constexpr int kNormE = 4;            // steps unrolled by the split and the short fused kernels
constexpr int kNormSplitThreads = 256;

// Elements per access: 16 bytes of the wider type, 8 at most; 4 in the
// backward, which keeps sums and scales of each channel.
constexpr int norm_max_vec(size_t xs, size_t ys, bool backward) { return xs == 2 && ys == 2 && !backward ? 8 : 4; }

// Steps whose values a thread of a 1024-thread block can hold: 128 registers,
// 64 of them for the values of x (forward) or of x and dy (backward), fewer
// where it keeps a group per channel as well, or where windows of y change
// layout. (16 steps of these spill, and a register that the compiler reloads
// in the block between a tile's loop and its barrier, where no lane is active
// yet, keeps what it held: an instance left windows unwritten so.)
constexpr int norm_max_steps(bool backward, bool straddle, bool cross) {
    return backward ? (straddle ? 4 : 8) : cross ? 8 : 16;
}

// One pass of the group norm. A block handles a slab of `slabC` channels (K
// whole groups, or 1/J of one) over `chunk` pixels of one image. With
// channels-last x a thread holds V adjacent channels of one pixel per step,
// `tc` threads across the slab and `tp` pixels per step; with NCHW x it holds V
// adjacent pixels of one channel, `tp` threads across the pixels and `tc`
// across the channels. A step covers `window` pixels of the slab's channels.
struct NormShape {
    int threads, V, K, J, slabC, nslab;
    int tc, tp, window;
    int steps;                // steps per block
    int split;                // 1: statistics and output in two kernels
    int chunk, nchunk;        // pixels per block, blocks along the pixels
    int tsteps;               // steps whose windows change layout together in LDS
};

// Floats of LDS that the kernels' sums take, without their results: a row of
// the vectors' values per thread (NHWC), and a value per thread or channel.
constexpr int norm_sum_floats(const NormShape &s, bool nhwc) {
    return (nhwc ? s.threads * s.V : 0) + (s.threads > s.slabC ? s.threads : s.slabC);
}

struct NormGeo {
    int N, C, P, G, cpg;
    float eps;
    int act;
    int64_t xs, ys;           // elements between pixels (NHWC)
    int x_nhwc, y_nhwc;
    NormShape f, b;           // forward, backward
};

struct NormPtrs {
    const void *x, *dy;
    const float *shift, *gamma, *beta;
    void *y, *dx;
    float *mean, *rstd;                  // forward: outputs (never NULL here)
    const float *mean_in, *rstd_in;      // backward
    float *dgamma, *dbeta, *dshift;      // may be NULL
    float *part;                         // forward, split: [N][G][nchunk J][2] mean, M2;
                                         // backward: [N][nchunk][3][C] sums over the pixels
    float *gpart;                        // backward, split: [N][G][nchunk J][2] group sums
    float *group;                        // backward, split: [N][G][2] group means
};

// By types: the kernels of each are compiled in a file of their own.
wq8_status launch_norm_forward_f32_f32(const NormGeo &g, const NormPtrs &p, void *stream);
wq8_status launch_norm_forward_f32_bf16(const NormGeo &g, const NormPtrs &p, void *stream);
wq8_status launch_norm_forward_bf16_f32(const NormGeo &g, const NormPtrs &p, void *stream);
wq8_status launch_norm_forward_bf16_bf16(const NormGeo &g, const NormPtrs &p, void *stream);
wq8_status launch_norm_backward_f32(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream);
wq8_status launch_norm_backward_bf16(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream);

// ---------------------------------------------------------- matrix product
// C[m][n] = sum_k A(m, k) B(n, k). An operand is stored with k contiguous
// (element (m, k) at m * ld + k) or with its rows' index contiguous
// (element (m, k) at k * ld + m).

// Block tile and the split of k over blocks of one product.
struct GemmShape {
    int tile;      // index into kGemmTiles
    int direct;    // whole k steps go from memory to LDS past the registers
    int splits;    // blocks along k; > 1: fp32 partial products, joined by a second kernel
    int ksteps;    // k steps per split
};

struct LinearGeo {
    int M, K, N;              // rows, Cin, Cout
    int act;
    int64_t xs, ys, rs;       // elements between rows of x, of y and of an NHWC residual
    int r_planar, pixels;
    GemmShape f, dx, dw;      // dx and dw share a tile: they run in one kernel
    int dz_own;               // backward: dz is written to the workspace (else it is dy itself)
    int dz_planes;            // 2: dz as the sum of two bf16 matrices
    int dz_chunk, dz_nchunk;  // rows per block of the dz kernel, blocks along the rows
};

struct LinearPtrs {
    const void *x, *w, *dy, *zin, *residual;
    const float *bias;
    void *y, *z, *dx, *dw;
    float *dbias;
    void *dz;                 // workspace: dz in x's type
    float *colsum;            // workspace: [dz_nchunk][N] column sums
    float *partial, *partial_dx, *partial_dw;  // workspace: split products
};

// The built tiles: rows, columns, blocks that a compute unit holds (of the
// kernels that load directly; by registers the backward's 128 x 128 holds one,
// 128 x 64 and 16 x 128 two), and the share of the largest tile's rate that a full card reaches in bf16 and in fp32
// (8192^3: 1337, 1150, 917 and 648 TFLOP/s in bf16; 8192 x 4096 x 4096: 146 to
// 140 in fp32). The last one is for a few rows.
struct GemmTile {
    int bm, bn, blocks;
    double bf16, f32;
};
constexpr GemmTile kGemmTiles[] = {
    {256, 256, 1, 1.0, 1.0}, {128, 128, 2, 0.86, 0.98}, {128, 64, 3, 0.69, 0.98}, {64, 64, 5, 0.49, 0.96}, {16, 128, 4, 0.3, 0.5}};
constexpr int kGemmTileCount = 5;

wq8_status launch_linear_forward_f32(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream);
wq8_status launch_linear_forward_bf16(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream);
wq8_status launch_linear_backward(const LinearGeo &g, wq8_dtype xdt, wq8_dtype ydt,
                                  const LinearPtrs &p, void *stream);

}  // namespace wq8

struct wq8_linear_plan {
    wq8::LinearGeo geo;
    wq8_dtype xdt, ydt;
    size_t f_off_partial, f_bytes;
    size_t b_off_dz, b_off_colsum, b_off_partial, b_off_partial_dw, b_bytes;
};

struct wq8_norm_plan {
    wq8::NormGeo geo;
    wq8_dtype xdt, ydt;
    size_t f_off_part, f_off_stats, f_bytes;           // forward workspace
    size_t b_off_part, b_off_group, b_off_gpart, b_bytes;  // backward workspace
};
