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
// and writes y (fused). Larger groups are split over blocks along the pixels
// into a statistics kernel, a small joining kernel and an output kernel that
// reads x again. Partial results are joined in a fixed order, without atomics.
//
// Layouts: threads follow the layout of x. When y (or dy) has the other
// layout each step's window of pixels x channels passes through LDS, so both
// sides access global memory along their contiguous dimension.
#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// ---------------------------------------------------------------- forward
template <typename XT, typename YT, int V, bool CL, bool CROSS, int E, int MODE>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormGeo g, NormPtrs a) {
    constexpr int NC = CL ? V : 1;
    extern __shared__ __align__(16) char smem[];
    float *red = (float *)smem;
    const NormShape &s = g.f;
    const Where w = locate<V, CL>(g, s);
    const XT *x = (const XT *)a.x;
    YT *y = (YT *)a.y;

    Vec<XT, V> f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (e < s.steps) {
            const int p = pixel_of<V, CL>(s, w, e);
            f[e] = load_vec_n<XT, V>(addr<XT, V, CL>(x, g, g.xs, w.n, w.c, p), count_of<V, CL>(w, p));
        }
    }
    float sh[NC];
    per_channel<V, CL>(sh, a.shift, (int64_t)w.n * g.C + w.c, w.on, 0.0f);

    float mean, rstd;
    if constexpr (MODE != kApply) {
        // members of this thread's group in the block
        const int chans = s.J == 1 ? g.cpg : w.cend - w.slab0;
        const float cnt = (float)(w.pend - w.p0) * (float)chans;
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < s.steps) {
                const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
                float u = 0.0f;
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k < n) u += to_f32(f[e].v[k]) + sh[CL ? k : 0];
                t += u;
            }
        mean = group_sum<V, CL>(t, g, s, w, red) / cnt;
        t = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < s.steps) {
                const int n = count_of<V, CL>(w, pixel_of<V, CL>(s, w, e));
                float u = 0.0f;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = to_f32(f[e].v[k]) + sh[CL ? k : 0] - mean;
                    if (k < n) u = fmaf(d, d, u);
                }
                t += u;
            }
        const float m2 = group_sum<V, CL>(t, g, s, w, red);
        // the first thread of each group writes what the group has
        const bool first = w.on && w.tp == 0 && (s.J > 1 ? w.tc == 0 : w.c == w.slab0 + w.kg * g.cpg);
        if constexpr (MODE == kReduce) {
            if (first) {
                const int64_t at = ((int64_t)w.n * g.G + w.g0 + w.kg) * (s.nchunk * s.J) + w.chunk * s.J + w.part;
                a.part[2 * at] = mean;
                a.part[2 * at + 1] = m2;
            }
            return;
        }
        rstd = 1.0f / sqrtf(m2 / cnt + g.eps);
        if (first) {
            const int64_t at = (int64_t)w.n * g.G + w.g0 + w.kg;
            a.mean[at] = mean;
            a.rstd[at] = rstd;
        }
    } else {
        const int64_t at = (int64_t)w.n * g.G + w.g0 + w.kg;
        mean = a.mean[at];
        rstd = a.rstd[at];
    }

    if constexpr (MODE != kReduce) {
        float ga[NC], be[NC];
        per_channel<V, CL>(ga, a.gamma, w.c, w.on, 1.0f);
        per_channel<V, CL>(be, a.beta, w.c, w.on, 0.0f);
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < s.steps) {
                    const int p = pixel_of<V, CL>(s, w, e), n = count_of<V, CL>(w, p);
                    Vec<YT, V> r;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const int kc = CL ? k : 0;
                        const float h = (to_f32(f[e].v[k]) + sh[kc] - mean) * rstd;
                        r.v[k] = from_f32<YT>(act_fwd<decltype(act)::value>(fmaf(h, ga[kc], be[kc])));
                    }
                    if constexpr (!CROSS) {
                        if (n > 0) store_vec_n<YT, V>((YT *)addr<YT, V, CL>(y, g, g.ys, w.n, w.c, p), r, n);
                    } else {
                        YT *tile = (YT *)smem;
                        if (w.on)
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

// Joins the partial statistics of a group (one wave): the mean of the parts'
// means weighted by their counts, then M2 = sum M2_i + n_i (mean_i - mean)^2.
__global__ __launch_bounds__(256) void k_norm_join(NormGeo g, NormPtrs a) {
    const NormShape &s = g.f;
    const int lane = threadIdx.x & 63;
    const int64_t ng = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (ng >= (int64_t)g.N * g.G) return;
    const int np = s.nchunk * s.J;
    const float *part = a.part + 2 * ng * np;
    const auto count = [&](int i) {
        const int ch = i / s.J, j = i % s.J;
        const int px = min(s.chunk, g.P - ch * s.chunk);
        const int c = s.J == 1 ? g.cpg : min(s.slabC, g.cpg - j * s.slabC);
        return (float)px * (float)c;
    };
    float t = 0.0f;
    for (int i = lane; i < np; i += 64) t = fmaf(count(i), part[2 * i], t);
    const float m = (float)((double)g.P * g.cpg);
    const float mean = wave_sum(t) / m;
    t = 0.0f;
    for (int i = lane; i < np; i += 64) {
        const float d = part[2 * i] - mean;
        t += fmaf(count(i) * d, d, part[2 * i + 1]);
    }
    t = wave_sum(t);
    if (lane == 0) {
        a.mean[ng] = mean;
        a.rstd[ng] = 1.0f / sqrtf(t / m + g.eps);
    }
}

struct RunForward {
    const NormGeo &g;
    const NormPtrs &p;
    hipStream_t st;

    template <typename XT, typename YT, int V, bool CL, bool CROSS, int E>
    void operator()() const {
        const NormShape &s = g.f;
        const dim3 grid((unsigned)((int64_t)g.N * s.nslab * s.nchunk)), blk(s.threads);
        const size_t red = reduce_lds(s, CL, false), tile = CROSS ? tile_lds<YT>(s, CL) : 0;
        const size_t both = red > tile ? red : tile;
        if (s.fused) {
            hipLaunchKernelGGL((k_norm_fwd<XT, YT, V, CL, CROSS, E, kFused>), grid, blk, both, st, g, p);
            return;
        }
        if constexpr (E == kNormE) {
            hipLaunchKernelGGL((k_norm_fwd<XT, XT, V, CL, false, E, kReduce>), grid, blk, red, st, g, p);
            hipLaunchKernelGGL(k_norm_join, dim3((unsigned)(((int64_t)g.N * g.G + 3) / 4)), dim3(256), 0, st, g, p);
            hipLaunchKernelGGL((k_norm_fwd<XT, YT, V, CL, CROSS, E, kApply>), grid, blk, tile, st, g, p);
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
