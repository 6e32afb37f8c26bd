// Backward of the group norm with an activation (see wq8_norm_fwd.hip for the
// mathematics, the split and the layouts).
#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// A block leaves the sums S1, S2, S3 of its channels over its pixels in
// `part`. Fused, it forms the group means from them and writes dx at once.
// Split, a first kernel leaves each group's weighted sums as well, and a second
// one joins those of its groups and writes dx. The parameters' gradients and
// dshift come from `part` in a last, small kernel.
template <typename XT, typename YT, int V, int KIND, bool CROSS, int E, int MODE>
__global__ __launch_bounds__(MODE == kFused ? 1024 : kNormSplitThreads) void k_norm_bwd(NormGeo g, NormPtrs a) {
    constexpr bool CL = KIND != kPlanar;
    constexpr int NC = CL ? V : 1, NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.b;
    float *const gm = (float *)smem, *const chan = gm + 2 * s.K, *const red = chan + 2 * s.slabC;
    const Where w = locate<V, CL>(g, s, xcd_block(blockIdx.x, gridDim.x));
    const XT *x = (const XT *)a.x;
    const YT *dy = (const YT *)a.dy;

    Vec<XT, V> fx[E];
    Vec<YT, V> fd[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < s.steps) {
            const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
            fx[e] = load_part<XT, V, KIND>(addr<XT, V, CL>(x, g, g.xs, w.n, w.c, p), n);
            if constexpr (!CROSS)
                fd[e] = load_part<YT, V, KIND>(addr<YT, V, CL>(dy, g, g.ys, w.n, w.c, p), n);
        }
    if constexpr (CROSS) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < s.steps) {
                YT *tile = (YT *)smem;
                global_to_tile<YT, CL>(tile, dy, g, s, w, g.ys, w.p0 + e * s.window);
                __syncthreads();
                const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
#pragma unroll
                for (int k = 0; k < V; ++k) fd[e].v[k] = k < n ? tile[tile_at<CL, V>(s, w, k)] : YT(0);
                __syncthreads();
            }
    }
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    float off[NC], ga[NC], be[NC], rstd[NG];
    per_channel<V, CL>(off, a.shift, (int64_t)w.n * g.C + w.c, w.nc, 0.0f);
    per_channel<V, CL>(ga, a.gamma, w.c, w.nc, 1.0f);
    per_channel<V, CL>(be, a.beta, w.c, w.nc, 0.0f);
#pragma unroll
    for (int k = 0; k < NC; ++k) off[k] -= a.mean_in[group0 + group_of<V, KIND>(g, s, w, k)];
#pragma unroll
    for (int k = 0; k < NG; ++k) rstd[k] = a.rstd_in[group0 + group_of<V, KIND>(g, s, w, k)];

    if constexpr (MODE != kApply) {
        float s1[NC] = {}, s2[NC] = {}, s3[NC] = {};
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < s.steps) {
                    const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const int kc = CL ? k : 0;
                        const float h = (to_f32(fx[e].v[k]) + off[kc]) * rstd[NG == 1 ? 0 : k];
                        const float dz = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value>(fmaf(h, ga[kc], be[kc]));
                        if (k < n) {
                            s1[kc] += dz;
                            s2[kc] = fmaf(dz, h, s2[kc]);
                            s3[kc] += h;
                        }
                    }
                }
        });
        if constexpr (MODE == kFused) {
            forget(fx);
            forget(fd);
        }
        float *const c1 = chan, *const c2 = chan + s.slabC;
        channel_sum<V, CL>(s1, s, w, red, c1);
        channel_sum<V, CL>(s2, s, w, red, c2);
        const auto weight = [&](int c) { return a.gamma ? a.gamma[w.slab0 + c] : 1.0f; };
        groups_of_channels(g, s, w, [&](int c) { return weight(c) * c1[c]; }, gm, 2);
        groups_of_channels(g, s, w, [&](int c) { return weight(c) * c2[c]; }, gm + 1, 2);
        float *out = a.part + ((int64_t)w.n * s.nchunk + w.chunk) * 3 * g.C + w.slab0;
        const int nc = w.cend - w.slab0;
        for (int c = threadIdx.x; c < nc; c += blockDim.x) {
            out[c] = c1[c];
            out[g.C + c] = c2[c];
        }
        __syncthreads();
        if (a.dshift) {
            channel_sum<V, CL>(s3, s, w, red, c1);
            for (int c = threadIdx.x; c < nc; c += blockDim.x) out[2 * (int64_t)g.C + c] = c1[c];
        }
        for (int k = threadIdx.x; k < 2 * s.K; k += blockDim.x) {
            if constexpr (MODE == kReduce) {
                const int64_t at = (group0 + k / 2) * (s.nchunk * s.J) + w.chunk * s.J + w.part;
                a.gpart[2 * at + k % 2] = gm[k];
            } else {
                a.group[2 * group0 + k] = gm[k] = gm[k] / (float)((double)g.P * g.cpg);
            }
        }
    } else {
        const int lane = threadIdx.x & 63, np = s.nchunk * s.J;
        for (int k = threadIdx.x >> 6; k < s.K; k += blockDim.x >> 6) {
            const float *part = a.gpart + 2 * (group0 + k) * np;
            float t1 = 0.0f, t2 = 0.0f;
            for (int i = lane; i < np; i += 64) {
                t1 += part[2 * i];
                t2 += part[2 * i + 1];
            }
            const float m = (float)((double)g.P * g.cpg);
            t1 = wave_sum(t1) / m;
            t2 = wave_sum(t2) / m;
            if (lane == 0) {
                gm[2 * k] = t1;
                gm[2 * k + 1] = t2;
                if (w.chunk == 0 && w.part == 0) {
                    a.group[2 * (group0 + k)] = t1;
                    a.group[2 * (group0 + k) + 1] = t2;
                }
            }
        }
    }

    if constexpr (MODE != kReduce) {
        __syncthreads();
        float m1[NG], m2[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            m1[k] = gm[2 * group_of<V, KIND>(g, s, w, k)];
            m2[k] = gm[2 * group_of<V, KIND>(g, s, w, k) + 1];
        }
        XT *dx = (XT *)a.dx;
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < s.steps) {
                    const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
                    Vec<XT, V> r;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const int kc = CL ? k : 0, kg = NG == 1 ? 0 : k;
                        const float h = (to_f32(fx[e].v[k]) + off[kc]) * rstd[kg];
                        const float dz = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value>(fmaf(h, ga[kc], be[kc]));
                        r.v[k] = from_f32<XT>(rstd[kg] * (fmaf(dz, ga[kc], -m1[kg]) - h * m2[kg]));
                    }
                    store_part<XT, V, KIND>((XT *)addr<XT, V, CL>(dx, g, g.xs, w.n, w.c, p), r, n);
                }
        });
    }
}

// dgamma, dbeta: sums of `part` over images and chunks; dshift of image n from
// its own: rstd (gamma S1 - P m1 - m2 S3). 16 channels a block, 16 lanes along
// the rows of `part`; block row y < N is an image's dshift, the last one the
// parameters' gradients.
__global__ __launch_bounds__(256) void k_norm_params(NormGeo g, NormPtrs a, int ncol, int only_params) {
    __shared__ float red[2][16][17];
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
    const int n = blockIdx.x / ncol, c = (blockIdx.x - n * ncol) * 16 + tc;
    const bool shift = !only_params && n < g.N;
    const int64_t row = 3 * (int64_t)g.C;
    const int64_t first = shift ? (int64_t)n * g.b.nchunk : 0;
    const int64_t last = shift ? first + g.b.nchunk : (int64_t)g.N * g.b.nchunk;
    float t1 = 0.0f, t2 = 0.0f;
    if (c < g.C) {
        const float *s1 = a.part + c, *s2 = s1 + (shift ? 2 * (int64_t)g.C : g.C);
        for (int64_t r = first + tr; r < last; r += 16) {
            t1 += s1[r * row];
            t2 += s2[r * row];
        }
    }
    red[0][tr][tc] = t1;
    red[1][tr][tc] = t2;
    __syncthreads();
    if (tr != 0 || c >= g.C) return;
    t1 = t2 = 0.0f;
    for (int i = 0; i < 16; ++i) {
        t1 += red[0][i][tc];
        t2 += red[1][i][tc];
    }
    if (shift) {
        const int64_t ng = (int64_t)n * g.G + c / g.cpg;
        const float gc = a.gamma ? a.gamma[c] : 1.0f;
        const float m1 = a.group[2 * ng], m2 = a.group[2 * ng + 1];
        a.dshift[(int64_t)n * g.C + c] = a.rstd_in[ng] * (fmaf(gc, t1, -(float)g.P * m1) - m2 * t2);
    } else {
        if (a.dbeta) a.dbeta[c] = t1;
        if (a.dgamma) a.dgamma[c] = t2;
    }
}

struct RunBackward {
    const NormGeo &g;
    const NormPtrs &p;
    hipStream_t st;

    template <typename XT, typename YT, int V, int KIND, bool CROSS, bool SPLIT, int E>
    void operator()() const {
        const NormShape &s = g.b;
        const dim3 grid((unsigned)((int64_t)g.N * s.nslab * s.nchunk)), blk(s.threads);
        const size_t red = (size_t)(2 * s.K + 2 * s.slabC + sum_floats(s, KIND)) * 4;
        const size_t tile = CROSS ? tile_lds<YT>(s, KIND != kPlanar) : 0;
        const size_t both = red > tile ? red : tile, own = (size_t)2 * s.K * 4;
        if constexpr (!SPLIT) {
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, KIND, CROSS, E, kFused>), grid, blk, both, st, g, p);
        } else {
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, KIND, CROSS, E, kReduce>), grid, blk, both, st, g, p);
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, KIND, CROSS, E, kApply>), grid, blk, own > tile ? own : tile, st,
                               g, p);
        }
    }
};

}  // namespace

wq8_status launch_norm_backward(const NormGeo &g, wq8_dtype xdt, wq8_dtype ydt, const NormPtrs &p,
                                void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (g.N > 0) pick_kernel<true>(g, xdt, ydt, RunBackward{g, p, st});
    if (p.dgamma || p.dbeta || (p.dshift && g.N > 0)) {
        const int ncol = (g.C + 15) / 16, rows = p.dshift ? g.N + 1 : 1;
        hipLaunchKernelGGL(k_norm_params, dim3((unsigned)((int64_t)ncol * rows)), dim3(256), 0, st, g, p, ncol, !p.dshift);
    }
    return check_launch("group norm backward");
}

}  // namespace wq8
