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
// layout windows of pixels x channels pass through LDS, so both sides access
// global memory along their contiguous dimension.
//
// Measured: 8 x 640 x 128 x 128 bf16 136 us: statistics 58 us (168 MB, 2.9 TB/s:
// 98 registers leave four blocks on a compute unit, and each ends in joins),
// output 77.5 us (336 MB, 4.3 TB/s, a large copy's rate is 4.7). 8 x 1280 x 16 x 16
// f32 NCHW 7.8 us fused (21 MB), 32 x 512 x 7 x 7 bf16 7 us, 2 x 320 x 64 x 64 bf16 to
// NCHW 18.4 us split (64 groups would leave three quarters of the card idle;
// fused they took 35 us): launch and load latency bound these three.
#pragma once

#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// ---------------------------------------------------------------- forward
// Mean and 1/sqrt(variance + eps) of the block's groups from all blocks' partial
// statistics, to gstat[K] and gstat[K..2K): the parts' means weighted by their
// counts, then M2 = sum M2_i + n_i (mean_i - mean)^2. A wave joins 4 groups at
// once, 128 parts of each at a time, with all their loads in flight.
__device__ __forceinline__ void join_stats(const NormGeo &g, const NormPtrs &a, int64_t group0, float *gstat) {
    constexpr int GB = 4, PB = 2;
    const NormShape &s = g.f;
    const int lane = threadIdx.x & 63, np = s.nchunk * s.J;
    const float m = (float)((double)g.P * g.cpg);
    const auto count = [&](int i) {
        if (i >= np) return 0.0f;
        const int ch = i / s.J, j = i - ch * s.J;
        const int px = min(s.chunk, g.P - ch * s.chunk);
        const int c = s.J == 1 ? g.cpg : min(s.slabC, g.cpg - j * s.slabC);
        return (float)px * (float)c;
    };
    for (int k0 = (threadIdx.x >> 6) * GB; k0 < s.K; k0 += kNormSplitThreads / 64 * GB) {
        Vec<float, 2> v[GB][PB];
        const auto fetch = [&](int i0) {
#pragma unroll
            for (int k = 0; k < GB; ++k)
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    v[k][i] = load_vec<float, 2>(a.part + 2 * ((group0 + min(k0 + k, s.K - 1)) * np + min(i0 + i * 64 + lane, np - 1)));
        };
        float t[GB] = {}, mean[GB];
        for (int i0 = 0; i0 < np; i0 += 64 * PB) {
            fetch(i0);
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const float n = count(i0 + i * 64 + lane);
#pragma unroll
                for (int k = 0; k < GB; ++k) t[k] += n > 0.0f ? n * v[k][i].v[0] : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < GB; ++k) {
            mean[k] = wave_sum(t[k]) / m;
            t[k] = 0.0f;
        }
        for (int i0 = 0; i0 < np; i0 += 64 * PB) {
            if (np > 64 * PB) fetch(i0);
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const float n = count(i0 + i * 64 + lane);
#pragma unroll
                for (int k = 0; k < GB; ++k) {
                    const float d = v[k][i].v[0] - mean[k];
                    t[k] += n > 0.0f ? fmaf(n * d, d, v[k][i].v[1]) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < GB; ++k) {
            const float r = 1.0f / sqrtf(wave_sum(t[k]) / m + g.eps);
            if (lane == 0 && k0 + k < s.K) {
                gstat[k0 + k] = mean[k];
                gstat[s.K + k0 + k] = r;
            }
        }
    }
}

// What remains of the fused and of the output kernel: z = (v - mean) rstd gamma
// + beta as one fma, the activation, and the vectors' way out. first: the step
// that f[0] holds. With the other layout on y's side all values come first:
// the tile's way out stands in the code once a step, not once a step and
// activation.
template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__device__ __forceinline__ void write_out(const Vec<XT, V> (&f)[E], const float *off, const float *sc, const float *be,
                                          const NormGeo &g, const Where &w, YT *y, int first, YT *tile) {
    constexpr bool CL = KIND != kPlanar;
    const NormShape &s = g.f;
    const auto value = [&](auto act, int e, int k) {
        const int kc = CL ? k : 0;
        return from_f32<YT>(act_fwd<decltype(act)::value, exact_acts<YT, YT>()>(fmaf(to_f32(f[e].v[k]) + off[kc], sc[kc], be[kc])));
    };
    if constexpr (!CROSS) {
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (first + e < s.steps) {
                    const Step at = step_of<V, KIND>(s, w, first + e);
                    Vec<YT, V> r;
#pragma unroll
                    for (int k = 0; k < V; ++k) r.v[k] = value(act, e, k);
                    if (at.lo < V) store_vec<YT, V>(addr<YT, V, KIND>(y, g, g.ys, w, at.p), r);
                }
        });
    } else {
        Vec<YT, V> r[E] = {};
        with_act(g.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (first + e < s.steps)
#pragma unroll
                    for (int k = 0; k < V; ++k) r[e].v[k] = value(act, e, k);
        });
        int te = 0;  // steps in the tile
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (first + e < s.steps) {
                const Step at = step_of<V, KIND>(s, w, first + e);
                const int p0 = w.p0 + (first + e - te) * s.window;
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k >= at.lo) tile[tile_at<V, KIND>(s, w, p0, at.p, k)] = r[e].v[k];
                if (++te == s.tsteps || e == E - 1 || first + e == s.steps - 1) {
                    __syncthreads();
                    tile_to_global<YT, CL>(tile, y, g, s, w, g.ys, p0);
                    __syncthreads();
                    te = 0;
                }
            }
    }
}

// off = shift - mean, sc = rstd gamma, be = beta of the thread's channels;
// gstat: the block's groups' means, then their rstd.
template <int V, int KIND>
__device__ __forceinline__ void scales(float *off, float *sc, float *be, const NormGeo &g, const NormPtrs &a, const Where &w,
                                       const float *gstat) {
    constexpr int NC = thread_channels<V, KIND>();
    const NormShape &s = g.f;
    per_channel<V, KIND>(sc, a.gamma, w.c, kOnes);
    per_channel<V, KIND>(be, a.beta, w.c, kZeros);
    int kg[NC];
    groups_of<V, KIND>(kg, g, s, w);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        off[k] -= gstat[kg[k]];
        sc[k] *= gstat[s.K + kg[k]];
    }
}

// One pass: a block holds its groups' values in registers.
template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__global__ __launch_bounds__(1024) void k_norm_fused(NormGeo g, NormPtrs a) {
    constexpr int NC = thread_channels<V, KIND>(), NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.f;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const red = (float *)smem, *const gstat = red + norm_sum_floats(s, KIND != kPlanar);  // means, then M2, then rstd
    const Where w = locate<V, KIND>(g, s, b);

    Vec<XT, V> f[E];
    load_steps<XT, V, KIND, E>(f, (const XT *)a.x, g, s, g.xs, w, 0);
    float off[NC];
    per_channel<V, KIND>(off, a.shift, (int64_t)w.n * g.C + w.c, kZeros);
    const float cnt = (float)((double)g.P * g.cpg);
    float t[NG] = {};
    for_values<V, KIND, E, false>(s, w, 0, [&](int e, int k, auto ok) {
        const float v = to_f32(f[e].v[k]) + off[NC == 1 ? 0 : k];
        t[NG == 1 ? 0 : k] += ok ? v : 0.0f;
    });
    drop_unowned<V, KIND>(w, t);
    group_sum<V, KIND>(t, g, s, w, red, gstat);
    if constexpr (!keeps_derived(V, E, KIND)) forget(f);
    int kg[NC];
    groups_of<V, KIND>(kg, g, s, w);
    float mean[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        mean[k] = gstat[kg[k]] / cnt;
        t[k] = 0.0f;
    }
    for_values<V, KIND, E, false>(s, w, 0, [&](int e, int k, auto ok) {
        const float v = to_f32(f[e].v[k]) + off[NC == 1 ? 0 : k] - mean[NG == 1 ? 0 : k], d = ok ? v : 0.0f;
        t[NG == 1 ? 0 : k] = fmaf(d, d, t[NG == 1 ? 0 : k]);
    });
    drop_unowned<V, KIND>(w, t);
    group_sum<V, KIND>(t, g, s, w, red, gstat + s.K);
    if constexpr (!keeps_derived(V, E, KIND)) forget(f);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    for (int k = threadIdx.x; k < s.K; k += blockDim.x) {
        a.mean[group0 + k] = gstat[k] = gstat[k] / cnt;
        a.rstd[group0 + k] = gstat[s.K + k] = 1.0f / sqrtf(gstat[s.K + k] / cnt + g.eps);
    }
    __syncthreads();
    float sc[NC], be[NC];
    scales<V, KIND>(off, sc, be, g, a, w, gstat);
    if constexpr (CROSS) __syncthreads();  // the tile takes the statistics' place
    write_out<XT, YT, V, KIND, CROSS, E>(f, off, sc, be, g, w, (YT *)a.y, 0, (YT *)smem);
}

// Split, first kernel: mean and M2 of each of the block's groups over its
// pixels. A thread sums d and d^2 of d = v - pivot, the pivot the mean of its
// own first B values. M2 = sum d^2 - (sum d)^2 / n then loses little however
// large the mean is: with the thread's true mean off the pivot by D, the first
// B values alone make M2 >= B D^2, so what is subtracted, n D^2, is at most
// n / B times the result. Threads are joined about the block's mean.
template <typename XT, int V, int KIND, int E>
__global__ __launch_bounds__(kNormSplitThreads) void k_norm_stats(NormGeo g, NormPtrs a) {
    constexpr int NC = thread_channels<V, KIND>(), NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.f;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const red = (float *)smem, *const gstat = red + norm_sum_floats(s, KIND != kPlanar);
    const Where w = locate<V, KIND>(g, s, b);
    float off[NC];
    per_channel<V, KIND>(off, a.shift, (int64_t)w.n * g.C + w.c, kZeros);

    // values per sum; by channel where a thread's channels are kept apart
    float have = 0.0f;
    float pivot[NG], s1[NG] = {}, s2[NG] = {};
    for (int first = 0; first < s.steps; first += E) {
        Vec<XT, V> f[E];
        load_steps<XT, V, KIND, E>(f, (const XT *)a.x, g, s, g.xs, w, first);
        float more = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int lo = step_of<V, KIND>(s, w, first + e).lo;
            more += KIND == kStraddle ? (lo < V ? 1.0f : 0.0f) : (float)(V - lo);
        }
        if (first == 0) {
            float t[NG] = {};
            for_values<V, KIND, E, true>(s, w, 0, [&](int e, int k, auto ok) {
                const float v = to_f32(f[e].v[k]) + off[NC == 1 ? 0 : k];
                t[NG == 1 ? 0 : k] += ok ? v : 0.0f;
            });
            const float inv = 1.0f / fmaxf(more, 1.0f);
#pragma unroll
            for (int k = 0; k < NG; ++k) pivot[k] = fabsf(t[k]) < INFINITY ? t[k] * inv : 0.0f;  // d of an infinity is that infinity
#pragma unroll
            for (int k = 0; k < NC; ++k) off[k] -= pivot[NG == 1 ? 0 : k];
        }
        have += more;
        for_values<V, KIND, E, true>(s, w, first, [&](int e, int k, auto ok) {
            const int kk = NG == 1 ? 0 : k;
            const float v = to_f32(f[e].v[k]) + off[NC == 1 ? 0 : k], d = ok ? v : 0.0f;
            s1[kk] += d;
            s2[kk] = fmaf(d, d, s2[kk]);
        });
    }
    const int chans = s.J == 1 ? g.cpg : w.cend - w.slab0;
    const float cnt = (float)(w.pend - w.p0) * (float)chans, inv = 1.0f / fmaxf(have, 1.0f);
    // nothing of what others own, in any value
    float t[NG], mean[NG], n[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        n[k] = KIND == kStraddle && k < w.lo ? 0.0f : have;
        mean[k] = fmaf(s1[k], inv, pivot[k]);
        t[k] = n[k] > 0.0f ? mean[k] * n[k] : 0.0f;
    }
    group_sum<V, KIND>(t, g, s, w, red, gstat);
    int kg[NC];
    groups_of<V, KIND>(kg, g, s, w);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        const float d = mean[k] - gstat[kg[k]] / cnt;
        const float m2 = fmaf(-s1[k], s1[k] * inv, s2[k]);
        t[k] = n[k] > 0.0f ? fmaf(d * d, n[k], m2) : 0.0f;
    }
    group_sum<V, KIND>(t, g, s, w, red, gstat + s.K);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    for (int k = threadIdx.x; k < s.K; k += blockDim.x) {
        const int64_t at = (group0 + k) * (s.nchunk * s.J) + w.chunk * s.J + w.part;
        a.part[2 * at] = gstat[k] / cnt;
        a.part[2 * at + 1] = gstat[s.K + k];
    }
}

// Split, second kernel: joins its groups' parts and writes y.
template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__global__ __launch_bounds__(kNormSplitThreads) void k_norm_apply(NormGeo g, NormPtrs a) {
    constexpr int NC = thread_channels<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.f;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const gstat = (float *)smem;
    const Where w = locate<V, KIND>(g, s, b);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    Vec<XT, V> f[E];
    load_steps<XT, V, KIND, E>(f, (const XT *)a.x, g, s, g.xs, w, 0);
    float off[NC], sc[NC], be[NC];
    per_channel<V, KIND>(off, a.shift, (int64_t)w.n * g.C + w.c, kZeros);
    join_stats(g, a, group0, gstat);
    __syncthreads();
    if (w.chunk == 0 && w.part == 0)
        for (int k = threadIdx.x; k < s.K; k += kNormSplitThreads) {
            a.mean[group0 + k] = gstat[k];
            a.rstd[group0 + k] = gstat[s.K + k];
        }
    scales<V, KIND>(off, sc, be, g, a, w, gstat);
    if constexpr (CROSS) __syncthreads();
    for (int first = 0;;) {
        write_out<XT, YT, V, KIND, CROSS, E>(f, off, sc, be, g, w, (YT *)a.y, first, (YT *)smem);
        first += E;
        if (first >= s.steps) break;
        load_steps<XT, V, KIND, E>(f, (const XT *)a.x, g, s, g.xs, w, first);
    }
}

struct RunForward {
    const NormGeo &g;
    const NormPtrs &p;
    hipStream_t st;

    template <typename XT, typename YT, int V, int KIND, bool CROSS, bool SPLIT, int E>
    void operator()() const {
        const NormShape &s = g.f;
        const dim3 grid = grid_of(norm_blocks(g, s)), blk(s.threads);
        const size_t red = (size_t)(2 * s.K + norm_sum_floats(s, KIND != kPlanar)) * 4, stats = (size_t)2 * s.K * 4;
        const size_t tile = CROSS ? tile_lds<YT>(s, KIND != kPlanar) : 0;
        if constexpr (!SPLIT) {
            hipLaunchKernelGGL((k_norm_fused<XT, YT, V, KIND, CROSS, E>), grid, blk, red > tile ? red : tile, st, g, p);
        } else {
            hipLaunchKernelGGL((k_norm_stats<XT, V, KIND, E>), grid, blk, red, st, g, p);
            hipLaunchKernelGGL((k_norm_apply<XT, YT, V, KIND, CROSS, E>), grid, blk, stats > tile ? stats : tile, st, g, p);
        }
    }
};

template <typename XT, typename YT>
wq8_status norm_forward(const NormGeo &g, const NormPtrs &p, void *stream) {
    pick_vector<false, XT, YT>(g, RunForward{g, p, (hipStream_t)stream});
    return check_launch("group norm");
}

}  // namespace
}  // namespace wq8
