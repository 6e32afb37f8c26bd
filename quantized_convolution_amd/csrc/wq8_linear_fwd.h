// Matrix product with bias, activation and residual: y = act(x w^T + bias) + residual.
//
// One kernel: the tiled product with everything after it in the epilogue, on
// the fp32 sums (8 adjacent columns of a row per thread: 16-byte stores of
// bf16). z, where the backward will want it, is rounded to y's type, as y is.
// An NCHW residual is read 16 adjacent pixels at a time. Measured: 16384 x 2560 x
// 10240 bf16 with gelu 807 to 833 us (1.05 PFLOP/s; the matrix cores bound it,
// the product alone takes a library 686 us), 8192 x 640 x 640 bf16 with a residual
// 15.2 us (32 MB; each block's start and end weigh as much as its 10 k steps),
// 2048 x 2560 x 1280 fp32 115 us (117 TFLOP/s; 105 and a join of 10), 8 x 320 x
// 1280 bf16 6.2 us (latency: the kernel takes 5, most of it launch, first loads
// and stores), 1 x 10240 x 10240 bf16 42 us (5.0 TB/s of weights).
#pragma once

#include "wq8_gemm_device.h"

namespace wq8 {
namespace {

static __device__ const float kNothing[8] = {};

template <typename YT>
struct EpiForward {
    const float *bias;
    const YT *residual;
    YT *y, *z;
    int64_t ys, rs;
    int M, N, act, planar, pixels;

    struct Column {
        Vec<float, 8> bias;
    };
    struct Item {
        Vec<YT, 8> residual;
    };

    // Rows and columns past the end read the last ones' values, and what is not
    // given reads zeros, so that loads stand under no condition but one for all.
    __device__ __forceinline__ Column column(int n) const {
        Column c;
        if (N % 8 == 0) c.bias = load_vec<float, 8>(bias ? bias + min(n, N - 8) : kNothing);
        else c.bias = load_vec_n<float, 8>(bias + n, bias ? N - n : 0);
        return c;
    }

    __device__ __forceinline__ Item item(int m, int n) const {
        Item r;
        const int row = min(m, M - 1);
        if (planar && residual) {
            const int img = row / pixels, p = row - img * pixels;
            const YT *src = residual + (int64_t)img * N * pixels + p;
#pragma unroll
            for (int e = 0; e < 8; ++e) r.residual.v[e] = src[(int64_t)min(n + e, N - 1) * pixels];
        } else if (N % 8 == 0) {
            r.residual = load_vec<YT, 8>(residual ? residual + row * rs + min(n, N - 8) : (const YT *)kNothing);
        } else {
            r.residual = load_vec_n<YT, 8>(residual + row * rs + n, residual ? N - n : 0);
        }
        return r;
    }

    template <typename F>
    __device__ __forceinline__ void with(F f) const {
        with_act(act, f);
    }

    template <int ACT>
    __device__ __forceinline__ void store(int m, int n, Vec<float, 8> v, int cnt, const Column &col, const Item &item) const {
        if (bias)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += col.bias.v[e];
        Vec<YT, 8> r;
        if (z) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
            store_vec_n<YT, 8>(z + (int64_t)m * N + n, r, cnt);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = act_fwd<ACT, exact_acts<YT, YT>()>(v.v[e]);
        if (residual)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += to_f32(item.residual.v[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
        store_vec_n<YT, 8>(y + (int64_t)m * ys + n, r, cnt);
    }
};

template <typename XT, typename YT>
struct RunForward {
    const LinearGeo &g;
    const LinearPtrs &p;
    hipStream_t st;

    template <int BM, int BN, int WM, int WN, bool DIRECT>
    void operator()() const {
        using EPI = EpiForward<YT>;
        const EPI epi = {p.bias, (const YT *)p.residual, (YT *)p.y, (YT *)p.z, g.ys, g.rs, g.M, g.N, g.act, g.r_planar,
                         g.pixels};
        GemmArgs a = {};
        a.A = p.x;
        a.B = p.w;
        a.lda = g.xs;
        a.ldb = g.K;
        a.M = g.M;
        a.N = g.N;
        a.K = g.K;
        const int64_t blocks = set_tiles<BM, BN>(a, g.f, p.partial);
        const auto kernel = k_gemm<XT, true, true, BM, BN, WM, WN, DIRECT, EPI>;
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(WM * WN * 64), (tile_lds<BM, BN>(kernel)), st, a, epi);
        if (a.splits > 1)
            hipLaunchKernelGGL((k_gemm_join<EPI>), grid_of(join_blocks(a)), dim3(256), 0, st, a, epi, (int)join_blocks(a));
    }
};

template <typename XT>
wq8_status linear_forward(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (ydt == WQ8_F32) pick_tile<false>(g.f, RunForward<XT, float>{g, p, st});
    else pick_tile<false>(g.f, RunForward<XT, bf16_t>{g, p, st});
    return check_launch("matrix product");
}

}  // namespace
}  // namespace wq8
