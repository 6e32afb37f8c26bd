// Matrix product with bias, activation and residual: y = act(x w^T + bias) + residual.
//
// One kernel: the tiled product with everything after it in the epilogue, on
// the fp32 sums (8 adjacent columns of a row per thread: 16-byte stores of
// bf16). z, where the backward will want it, is rounded to y's type, as y is.
// An NCHW residual is read 16 adjacent pixels at a time. Measured: 16384 x 2560 x
// 10240 bf16 with gelu 819 us (1.05 PFLOP/s; the matrix cores bound it, the
// product alone takes a library 686 us), 8192 x 640 x 640 bf16 with a residual
// 15.9 us (32 MB; each block's start and end weigh as much as its 10 k steps),
// 2048 x 2560 x 1280 fp32 116 us (116 TFLOP/s), 8 x 320 x 1280 bf16 6.1 us
// (latency: the kernel takes 5, most of it launch, first loads and stores).
#pragma once

#include "wq8_gemm_device.h"

namespace wq8 {
namespace {

template <typename YT>
struct EpiForward {
    const float *bias;
    const YT *residual;
    YT *y, *z;
    int64_t ys, rs;
    int N, act, planar, pixels;

    template <typename EACH>
    __device__ __forceinline__ void run(EACH each) const {
        with_act(act, [&](auto a) {
            each([&](int m, int n, Vec<float, 8> v, int cnt) { one<decltype(a)::value>(m, n, v, cnt); });
        });
    }

    template <int ACT>
    __device__ __forceinline__ void one(int m, int n, Vec<float, 8> v, int cnt) const {
        if (bias) {
            const Vec<float, 8> b = load_vec_n<float, 8>(bias + n, cnt);
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += b.v[e];
        }
        Vec<YT, 8> r;
        if (z) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
            store_vec_n<YT, 8>(z + (int64_t)m * N + n, r, cnt);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = act_fwd<ACT>(v.v[e]);
        if (residual) {
            if (planar) {
                const int img = m / pixels, p = m - img * pixels;
                const YT *src = residual + ((int64_t)img * N + n) * pixels + p;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < cnt) v.v[e] += to_f32(src[(int64_t)e * pixels]);
            } else {
                const Vec<YT, 8> s = load_vec_n<YT, 8>(residual + (int64_t)m * rs + n, cnt);
#pragma unroll
                for (int e = 0; e < 8; ++e) v.v[e] += to_f32(s.v[e]);
            }
        }
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
        const EPI epi = {p.bias, (const YT *)p.residual, (YT *)p.y, (YT *)p.z, g.ys, g.rs, g.N, g.act, g.r_planar, g.pixels};
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
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(WM * WN * 64), (tile_lds<BM, BN>(kernel)), st, a, epi);
        if (a.splits > 1)
            hipLaunchKernelGGL((k_gemm_join<EPI>), dim3((unsigned)join_blocks(a)), dim3(256), 0, st, a, epi);
    }
};

template <typename XT>
wq8_status linear_forward(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (ydt == WQ8_F32) pick_tile(g.f, RunForward<XT, float>{g, p, st});
    else pick_tile(g.f, RunForward<XT, bf16_t>{g, p, st});
    return check_launch("matrix product");
}

}  // namespace
}  // namespace wq8
