// Backward of the group norm with an activation (see wq8_norm_fwd.hip for the
// mathematics, the split and the layouts).
#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// --------------------------------------------------------------- backward
template <typename XT, typename YT, int V, bool CL, bool CROSS, int E, int MODE>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormGeo g, NormPtrs a) {
    constexpr int NC = CL ? V : 1;
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.b;
    const Where w = locate<V, CL>(g, s);
    const XT *x = (const XT *)a.x;
    const YT *dy = (const YT *)a.dy;

    Vec<XT, V> fx[E];
    Vec<YT, V> fd[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < s.steps) {
            const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
            fx[e] = load_vec_n<XT, V>(addr<XT, V, CL>(x, g, g.xs, w.n, w.c, p), n);
            if constexpr (!CROSS)
                fd[e] = load_vec_n<YT, V>(addr<YT, V, CL>(dy, g, g.ys, w.n, w.c, p), n);
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
    float sh[NC], ga[NC], be[NC];
    per_channel<V, CL>(sh, a.shift, (int64_t)w.n * g.C + w.c, w.on, 0.0f);
    per_channel<V, CL>(ga, a.gamma, w.c, w.on, 1.0f);
    per_channel<V, CL>(be, a.beta, w.c, w.on, 0.0f);
    const int64_t gat = (int64_t)w.n * g.G + w.g0 + w.kg;
    const float mean = a.mean_in[gat], rstd = a.rstd_in[gat];

    float m1, m2;
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
                        const float h = (to_f32(fx[e].v[k]) + sh[kc] - mean) * rstd;
                        const float dz = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value>(fmaf(h, ga[kc], be[kc]));
                        if (k < n) {
                            s1[kc] += dz;
                            s2[kc] = fmaf(dz, h, s2[kc]);
                            s3[kc] += h;
                        }
                    }
                }
        });
        float *rows = (float *)smem;
        float *rows2 = rows + (CL ? blockDim.x * V : 0);
        float *c1 = rows2 + max((int)blockDim.x, s.slabC), *c2 = c1 + s.slabC, *c3 = c2 + s.slabC;
        channel_sum<V, CL>(s1, s, w, rows, rows2, c1);
        channel_sum<V, CL>(s2, s, w, rows, rows2, c2);
        if (a.dshift) channel_sum<V, CL>(s3, s, w, rows, rows2, c3);
        const int nc = w.cend - w.slab0;
        if constexpr (MODE == kReduce) {
            float *out = a.part + ((int64_t)w.n * s.nchunk + w.chunk) * 3 * g.C + w.slab0;
            for (int c = threadIdx.x; c < nc; c += blockDim.x) {
                out[c] = c1[c];
                out[g.C + c] = c2[c];
                out[2 * (int64_t)g.C + c] = a.dshift ? c3[c] : 0.0f;
            }
            return;
        } else {
            // group means from the channels' sums: one wave per group
            float *gm = c3 + s.slabC;
            const int lane = threadIdx.x & 63;
            const float inv = 1.0f / (float)((double)g.P * g.cpg);
            for (int k = threadIdx.x >> 6; k < s.K; k += blockDim.x >> 6) {
                float t1 = 0.0f, t2 = 0.0f;
                for (int i = lane; i < g.cpg; i += 64) {
                    const int c = k * g.cpg + i;
                    const float gc = a.gamma ? a.gamma[w.slab0 + c] : 1.0f;
                    t1 = fmaf(gc, c1[c], t1);
                    t2 = fmaf(gc, c2[c], t2);
                }
                t1 = wave_sum(t1);
                t2 = wave_sum(t2);
                if (lane == 0) {
                    gm[2 * k] = t1 * inv;
                    gm[2 * k + 1] = t2 * inv;
                }
            }
            __syncthreads();
            m1 = gm[2 * w.kg];
            m2 = gm[2 * w.kg + 1];
            const int64_t nc0 = (int64_t)w.n * g.C + w.slab0, plane = (int64_t)g.N * g.C;
            for (int c = threadIdx.x; c < nc; c += blockDim.x) {
                a.sums[nc0 + c] = c1[c];
                a.sums[plane + nc0 + c] = c2[c];
                if (a.dshift) {
                    const int k = c / g.cpg;
                    const float gc = a.gamma ? a.gamma[w.slab0 + c] : 1.0f;
                    const float r = a.rstd_in[(int64_t)w.n * g.G + w.g0 + k];
                    a.dshift[nc0 + c] = r * (fmaf(gc, c1[c], -(float)g.P * gm[2 * k]) - gm[2 * k + 1] * c3[c]);
                }
            }
        }
    } else {
        m1 = a.group[2 * gat];
        m2 = a.group[2 * gat + 1];
    }

    if constexpr (MODE != kReduce) {
        XT *dx = (XT *)a.dx;
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < s.steps) {
                    const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
                    Vec<XT, V> r;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const int kc = CL ? k : 0;
                        const float h = (to_f32(fx[e].v[k]) + sh[kc] - mean) * rstd;
                        const float dz = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value>(fmaf(h, ga[kc], be[kc]));
                        r.v[k] = from_f32<XT>(rstd * (fmaf(dz, ga[kc], -m1) - h * m2));
                    }
                    if (n > 0) store_vec_n<XT, V>((XT *)addr<XT, V, CL>(dx, g, g.xs, w.n, w.c, p), r, n);
                }
        });
    }
}

// Joins the split backward's partial sums: a block per (image, group), a wave
// per channel over the chunks, then the group means.
__global__ __launch_bounds__(256) void k_norm_bwd_join(NormGeo g, NormPtrs a) {
    __shared__ float acc[4][2];
    const NormShape &s = g.b;
    const int64_t ng = blockIdx.x;
    const int n = (int)(ng / g.G), gr = (int)(ng % g.G);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t plane = (int64_t)g.N * g.C, step = 3 * (int64_t)g.C;
    const float r = a.rstd_in[ng], inv = 1.0f / (float)((double)g.P * g.cpg);
    float t1 = 0.0f, t2 = 0.0f;
    for (int i = wave; i < g.cpg; i += 4) {
        const int c = gr * g.cpg + i;
        const float *part = a.part + (int64_t)n * s.nchunk * step + c;
        float u1 = 0.0f, u2 = 0.0f;
        for (int k = lane; k < s.nchunk; k += 64) {
            u1 += part[k * step];
            u2 += part[k * step + g.C];
        }
        u1 = wave_sum(u1);
        u2 = wave_sum(u2);
        if (lane == 0) {
            a.sums[(int64_t)n * g.C + c] = u1;
            a.sums[plane + (int64_t)n * g.C + c] = u2;
        }
        const float gc = a.gamma ? a.gamma[c] : 1.0f;
        t1 = fmaf(gc, u1, t1);
        t2 = fmaf(gc, u2, t2);
    }
    if (lane == 0) {
        acc[wave][0] = t1;
        acc[wave][1] = t2;
    }
    __syncthreads();
    const float m1 = (acc[0][0] + acc[1][0] + acc[2][0] + acc[3][0]) * inv;
    const float m2 = (acc[0][1] + acc[1][1] + acc[2][1] + acc[3][1]) * inv;
    if (threadIdx.x == 0) {
        a.group[2 * ng] = m1;
        a.group[2 * ng + 1] = m2;
    }
    if (a.dshift)
        for (int i = wave; i < g.cpg; i += 4) {
            const int c = gr * g.cpg + i;
            const float *part = a.part + (int64_t)n * s.nchunk * step + c;
            float u3 = 0.0f;
            for (int k = lane; k < s.nchunk; k += 64) u3 += part[k * step + 2 * (int64_t)g.C];
            u3 = wave_sum(u3);
            // written by this wave above: channel c is wave's in both loops
            if (lane == 0) {
                const float gc = a.gamma ? a.gamma[c] : 1.0f;
                const float u1 = a.sums[(int64_t)n * g.C + c];
                a.dshift[(int64_t)n * g.C + c] = r * (fmaf(gc, u1, -(float)g.P * m1) - m2 * u3);
            }
        }
}

// dgamma, dbeta: sums over the images, 16 channels x 16 image lanes a block.
__global__ __launch_bounds__(256) void k_norm_params(NormGeo g, NormPtrs a) {
    __shared__ float red[2][16][17];
    const int tc = threadIdx.x & 15, tn = threadIdx.x >> 4, c = blockIdx.x * 16 + tc;
    float t1 = 0.0f, t2 = 0.0f;
    if (c < g.C)
        for (int n = tn; n < g.N; n += 16) {
            t1 += a.sums[(int64_t)n * g.C + c];
            t2 += a.sums[(int64_t)(g.N + n) * g.C + c];
        }
    red[0][tn][tc] = t1;
    red[1][tn][tc] = t2;
    __syncthreads();
    if (tn < 2 && c < g.C) {
        float t = 0.0f;
        for (int i = 0; i < 16; ++i) t += red[tn][i][tc];
        float *out = tn == 0 ? a.dbeta : a.dgamma;
        if (out) out[c] = t;
    }
}

struct RunBackward {
    const NormGeo &g;
    const NormPtrs &p;
    hipStream_t st;

    template <typename XT, typename YT, int V, bool CL, bool CROSS, int E>
    void operator()() const {
        const NormShape &s = g.b;
        const dim3 grid((unsigned)((int64_t)g.N * s.nslab * s.nchunk)), blk(s.threads);
        const size_t red = reduce_lds(s, CL, true), tile = CROSS ? tile_lds<YT>(s, CL) : 0;
        const size_t both = red > tile ? red : tile;
        if (s.fused) {
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, CL, CROSS, E, kFused>), grid, blk, both, st, g, p);
        } else if constexpr (E == kNormE) {
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, CL, CROSS, E, kReduce>), grid, blk, both, st, g, p);
            hipLaunchKernelGGL(k_norm_bwd_join, dim3((unsigned)((int64_t)g.N * g.G)), dim3(256), 0, st, g, p);
            hipLaunchKernelGGL((k_norm_bwd<XT, YT, V, CL, CROSS, E, kApply>), grid, blk, tile, st, g, p);
        }
    }
};

}  // namespace

wq8_status launch_norm_backward(const NormGeo &g, wq8_dtype xdt, wq8_dtype ydt, const NormPtrs &p,
                                void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (g.N > 0) pick_kernel<true>(g, xdt, ydt, RunBackward{g, p, st});
    if (p.dgamma || p.dbeta)
        hipLaunchKernelGGL(k_norm_params, dim3((g.C + 15) / 16), dim3(256), 0, st, g, p);
    return check_launch("group norm backward");
}

}  // namespace wq8
