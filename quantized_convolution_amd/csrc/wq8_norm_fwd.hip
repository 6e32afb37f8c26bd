// Group normalisation with an activation, forward and backward, on either
// activation layout.
//
// Mathematics: two-pass statistics (the mean first, then the squared
// deviations from it), held per thread, joined per group in fp32; the
// backward needs three sums per (image, channel) over the pixels,
//   S1 = sum dz,  S2 = sum dz h,  S3 = sum h,
// from which dbeta, dgamma, the two group means m1 = mean(gamma dz),
// m2 = mean(gamma dz h) and dshift = rstd (gamma S1 - P m1 - m2 S3) follow.
//
// What bounds it: memory. One element costs 10 to 25 operations for 4 to 12
// bytes moved, so a pass that reads and writes each tensor once is at its
// floor. Where a block can hold a whole group (up to 128 K bf16 values in the
// registers of 1024 threads) one kernel reads x once, reduces in the block
// and writes y (fused). Larger groups, and batches with too few groups to fill
// the card, are split over blocks along the pixels: a statistics kernel, then
// an output kernel that joins the parts of its groups and reads x again.
// Partial results are joined in a fixed order, without atomics.
//
// Layouts: threads follow the layout of x. When y (or dy) has the other
// layout each step's window of pixels x channels passes through LDS, so both
// sides access global memory along their contiguous dimension.
#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// ---------------------------------------------------------------- forward
// Mean and 1/sqrt(variance + eps) of group ng from its blocks' partial
// statistics (one wave): the parts' means weighted by their counts, then
// M2 = sum M2_i + n_i (mean_i - mean)^2.
__device__ __forceinline__ void join_stats(const NormGeo &g, const NormPtrs &a, int64_t ng, float &mean, float &rstd) {
    const NormShape &s = g.f;
    const int lane = threadIdx.x & 63, np = s.nchunk * s.J;
    const float *part = a.part + 2 * ng * np;
    const auto count = [&](int i) {
        const int ch = i / s.J, j = i - ch * s.J;
        const int px = min(s.chunk, g.P - ch * s.chunk);
        const int c = s.J == 1 ? g.cpg : min(s.slabC, g.cpg - j * s.slabC);
        return (float)px * (float)c;
    };
    float t = 0.0f;
    for (int i = lane; i < np; i += 64) t = fmaf(count(i), part[2 * i], t);
    const float m = (float)((double)g.P * g.cpg);
    mean = wave_sum(t) / m;
    t = 0.0f;
    for (int i = lane; i < np; i += 64) {
        const float d = part[2 * i] - mean;
        t += fmaf(count(i) * d, d, part[2 * i + 1]);
    }
    rstd = 1.0f / sqrtf(wave_sum(t) / m + g.eps);
}

template <typename XT, typename YT, int V, int KIND, bool CROSS, int E, int MODE>
__global__ __launch_bounds__(MODE == kFused ? 1024 : kNormSplitThreads) void k_norm_fwd(NormGeo g, NormPtrs a) {
    constexpr bool CL = KIND != kPlanar;
    constexpr int NC = CL ? V : 1, NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.f;
    float *const gstat = (float *)smem, *const red = gstat + 2 * s.K;  // means, then M2 or rstd
    const Where w = locate<V, CL>(g, s, xcd_block(blockIdx.x, gridDim.x));
    const XT *x = (const XT *)a.x;
    YT *y = (YT *)a.y;

    Vec<XT, V> f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e < s.steps) {
            const int p = pixel_of<V, CL>(s, w, e);
            f[e] = load_part<XT, V, KIND>(addr<XT, V, CL>(x, g, g.xs, w.n, w.c, p), count_of<V, CL>(w, p));
        }
    }
    float off[NC];  // shift, later shift - mean
    per_channel<V, CL>(off, a.shift, (int64_t)w.n * g.C + w.c, w.nc, 0.0f);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;

    if constexpr (MODE != kApply) {
        // values of a group in the block
        const int chans = s.J == 1 ? g.cpg : w.cend - w.slab0;
        const float cnt = (float)(w.pend - w.p0) * (float)chans;
        float t[NG] = {};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < s.steps) {
                const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k < n) t[NG == 1 ? 0 : k] += to_f32(f[e].v[k]) + off[CL ? k : 0];
            }
        group_sum<V, KIND>(t, g, s, w, red, gstat);
        forget(f);
        float mean[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) mean[k] = gstat[group_of<V, KIND>(g, s, w, k)] / cnt;
#pragma unroll
        for (int k = 0; k < NG; ++k) t[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < s.steps) {
                const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = to_f32(f[e].v[k]) + off[CL ? k : 0] - mean[NG == 1 ? 0 : k];
                    if (k < n) t[NG == 1 ? 0 : k] = fmaf(d, d, t[NG == 1 ? 0 : k]);
                }
            }
        group_sum<V, KIND>(t, g, s, w, red, gstat + s.K);
        if constexpr (MODE == kFused) forget(f);
        for (int k = threadIdx.x; k < s.K; k += blockDim.x) {
            const float mu = gstat[k] / cnt, m2 = gstat[s.K + k];
            if constexpr (MODE == kReduce) {
                const int64_t at = (group0 + k) * (s.nchunk * s.J) + w.chunk * s.J + w.part;
                a.part[2 * at] = mu;
                a.part[2 * at + 1] = m2;
            } else {
                a.mean[group0 + k] = gstat[k] = mu;
                a.rstd[group0 + k] = gstat[s.K + k] = 1.0f / sqrtf(m2 / cnt + g.eps);
            }
        }
    } else {
        for (int k = threadIdx.x >> 6; k < s.K; k += blockDim.x >> 6) {
            float mu, r;
            join_stats(g, a, group0 + k, mu, r);
            if ((threadIdx.x & 63) == 0) {
                gstat[k] = mu;
                gstat[s.K + k] = r;
                if (w.chunk == 0 && w.part == 0) {
                    a.mean[group0 + k] = mu;
                    a.rstd[group0 + k] = r;
                }
            }
        }
    }

    if constexpr (MODE != kReduce) {
        __syncthreads();
        float sc[NC], be[NC];
        per_channel<V, CL>(sc, a.gamma, w.c, w.nc, 1.0f);
        per_channel<V, CL>(be, a.beta, w.c, w.nc, 0.0f);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int gk = group_of<V, KIND>(g, s, w, k);
            off[k] -= gstat[gk];
            sc[k] *= gstat[s.K + gk];
        }
        if constexpr (CROSS) __syncthreads();  // the tile takes the statistics' place
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < s.steps) {
                    const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
                    Vec<YT, V> r;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const int kc = CL ? k : 0;
                        const float z = fmaf(to_f32(f[e].v[k]) + off[kc], sc[kc], be[kc]);
                        r.v[k] = from_f32<YT>(act_fwd<decltype(act)::value>(z));
                    }
                    if constexpr (!CROSS) {
                        store_part<YT, V, KIND>((YT *)addr<YT, V, CL>(y, g, g.ys, w.n, w.c, p), r, n);
                    } else {
                        YT *tile = (YT *)smem;
                        if (w.nc)
#pragma unroll
                            for (int k = 0; k < V; ++k) tile[tile_at<CL, V>(s, w, k)] = r.v[k];
                        __syncthreads();
                        tile_to_global<YT, CL>(tile, y, g, s, w, g.ys, w.p0 + e * s.window);
                        __syncthreads();
                    }
                }
        });
    }
}

struct RunForward {
    const NormGeo &g;
    const NormPtrs &p;
    hipStream_t st;

    template <typename XT, typename YT, int V, int KIND, bool CROSS, bool SPLIT, int E>
    void operator()() const {
        const NormShape &s = g.f;
        const dim3 grid((unsigned)((int64_t)g.N * s.nslab * s.nchunk)), blk(s.threads);
        const size_t red = (size_t)(2 * s.K + sum_floats(s, KIND) + (KIND == kStraddle ? s.slabC : 0)) * 4;
        const size_t tile = CROSS ? tile_lds<YT>(s, KIND != kPlanar) : 0;
        const size_t both = red > tile ? red : tile, own = (size_t)2 * s.K * 4;
        if constexpr (!SPLIT) {
            hipLaunchKernelGGL((k_norm_fwd<XT, YT, V, KIND, CROSS, E, kFused>), grid, blk, both, st, g, p);
        } else {
            hipLaunchKernelGGL((k_norm_fwd<XT, XT, V, KIND, false, E, kReduce>), grid, blk, red, st, g, p);
            hipLaunchKernelGGL((k_norm_fwd<XT, YT, V, KIND, CROSS, E, kApply>), grid, blk, own > tile ? own : tile, st,
                               g, p);
        }
    }
};

}  // namespace

wq8_status launch_norm_forward(const NormGeo &g, wq8_dtype xdt, wq8_dtype ydt, const NormPtrs &p,
                               void *stream) {
    pick_kernel<false>(g, xdt, ydt, RunForward{g, p, (hipStream_t)stream});
    return check_launch("group norm");
}

}  // namespace wq8
