// Backward of the group norm with an activation (see wq8_norm_fwd.h for the
// mathematics, the split and the layouts).
//
// x and dy are read once where a block holds a group (half as many values as
// forward: two tensors share the registers), else twice. Measured: 8 x 640 x 32 x 32
// bf16 fused 18.5 us (31 MB; the activation's slope, two quarter-rate
// instructions a value, is evaluated for the sums and again for dx: half of the
// kernel's 17 us is arithmetic), 2 x 320 x 64 x 64 f32 with dy in NCHW split 28.5 us in
// kernels of 14, 10 and 5.5 us (52 MB), 8 x 640 x 128 x 128 bf16 225 us (503 MB).
#pragma once

#include "wq8_norm_device.h"

namespace wq8 {
namespace {

// A block leaves the sums S1, S2, S3 of its channels over its pixels in
// `part`. Fused, it forms the group means from them and writes dx at once.
// Split, a first kernel leaves each group's weighted sums as well, and a second
// one joins those of its groups and writes dx. The parameters' gradients and
// dshift come from `part` in a last, small kernel.

// What a thread knows of its channels.
template <int V, int KIND>
struct Channels {
    static constexpr int NC = thread_channels<V, KIND>(), NG = group_values<V, KIND>();
    float off[NC], ga[NC], sc[NC], be[NC], rstd[NG];  // off = shift - mean, sc = gamma rstd
    int kg[NC];

    // z of v = x + off, in the forward's operations: relu's mask is the forward's
    __device__ __forceinline__ float z(float v, int k) const { return fmaf(v, sc[k], be[k]); }

    __device__ __forceinline__ void load(const NormGeo &g, const NormPtrs &a, const Where &w) {
        const int64_t group0 = (int64_t)w.n * g.G + w.g0;
        per_channel<V, KIND>(off, a.shift, (int64_t)w.n * g.C + w.c, kZeros);
        per_channel<V, KIND>(ga, a.gamma, w.c, kOnes);
        per_channel<V, KIND>(be, a.beta, w.c, kZeros);
        groups_of<V, KIND>(kg, g, g.b, w);
#pragma unroll
        for (int k = 0; k < NC; ++k) off[k] -= a.mean_in[group0 + kg[k]];
#pragma unroll
        for (int k = 0; k < NG; ++k) rstd[k] = a.rstd_in[group0 + kg[k]];
#pragma unroll
        for (int k = 0; k < NC; ++k) sc[k] = ga[k] * rstd[NG == 1 ? 0 : k];
    }
};

// dy of E steps from step `first`; with the other layout by way of LDS, zeros
// for what others own (ends with a barrier).
template <typename YT, int V, int KIND, bool CROSS, int E>
__device__ __forceinline__ void load_dy(Vec<YT, V> (&f)[E], const YT *dy, const NormGeo &g, const Where &w, int first, YT *tile) {
    constexpr bool CL = KIND != kPlanar;
    const NormShape &s = g.b;
    if constexpr (!CROSS) {
        load_steps<YT, V, KIND, E>(f, dy, g, s, g.ys, w, first);
    } else {
        int te = 0;  // steps read from the tile
#pragma unroll
        for (int e = 0; e < E; ++e) {
            f[e] = {};
            if (first + e < s.steps) {  // uniform: the tile's barriers
                if (te == 0) {
                    if (e > 0) __syncthreads();
                    global_to_tile<YT, CL>(tile, dy, g, s, w, g.ys, w.p0 + (first + e) * s.window);
                    __syncthreads();
                }
                const Step at = step_of<V, KIND>(s, w, first + e);
                const int p0 = w.p0 + (first + e - te) * s.window;
#pragma unroll
                for (int k = 0; k < V; ++k) f[e].v[k] = k >= at.lo ? tile[tile_at<V, KIND>(s, w, p0, at.p, k)] : YT(0);
                if (++te == s.tsteps) te = 0;
            }
        }
        __syncthreads();
    }
}

// Adds the steps' dz, dz h and h to the thread's sums.
template <typename XT, typename YT, int V, int KIND, int E, bool BATCH>
__device__ __forceinline__ void add_sums(float *s1, float *s2, float *s3, const Vec<XT, V> (&fx)[E], const Vec<YT, V> (&fd)[E],
                                         const Channels<V, KIND> &c, const NormGeo &g, const Where &w, int first) {
    with_act(g.act, [&](auto act) {
        for_values<V, KIND, E, BATCH>(g.b, w, first, [&](int e, int k, auto ok) {
            const int kc = c.NC == 1 ? 0 : k;
            const float v = to_f32(fx[e].v[k]) + c.off[kc], hv = v * c.rstd[c.NG == 1 ? 0 : k], h = ok ? hv : 0.0f;
            const float dv = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value, exact_acts<XT, YT>()>(c.z(v, kc));
            const float dz = ok ? dv : 0.0f;
            s1[kc] += dz;
            s2[kc] = fmaf(dz, h, s2[kc]);
            s3[kc] += h;
        });
    });
}

// Joins the threads' sums: the channels' into `part`, the groups' weighted
// totals into gm[2 K].
template <int V, int KIND>
__device__ __forceinline__ void join_sums(const NormGeo &g, const NormPtrs &a, const Where &w,
                                          float (&s1)[Channels<V, KIND>::NC], float (&s2)[Channels<V, KIND>::NC],
                                          float (&s3)[Channels<V, KIND>::NC], float *red, float *gm) {
    constexpr bool CL = KIND != kPlanar;
    const NormShape &s = g.b;
    float *const c1 = gm + 2 * s.K, *const c2 = c1 + s.slabC;
    drop_unowned<V, KIND>(w, s1);
    drop_unowned<V, KIND>(w, s2);
    drop_unowned<V, KIND>(w, s3);
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
}

// dx of the steps, gm: the groups' means of gamma dz and of gamma dz h.
template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__device__ __forceinline__ void write_dx(const Vec<XT, V> (&fx)[E], const Vec<YT, V> (&fd)[E], const Channels<V, KIND> &c,
                                         const float (&m1)[Channels<V, KIND>::NG], const float (&m2)[Channels<V, KIND>::NG],
                                         const NormGeo &g, const Where &w, XT *dx, int first) {
    constexpr bool CL = KIND != kPlanar;
    const NormShape &s = g.b;
    with_act(g.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (first + e < s.steps) {
                const Step at = step_of<V, KIND>(s, w, first + e);
                Vec<XT, V> r;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int kc = CL ? k : 0, kk = c.NG == 1 ? 0 : k;
                    const float v = to_f32(fx[e].v[k]) + c.off[kc], h = v * c.rstd[kk];
                    const float dz = to_f32(fd[e].v[k]) * act_slope<decltype(act)::value, exact_acts<XT, YT>()>(c.z(v, kc));
                    r.v[k] = from_f32<XT>(c.rstd[kk] * (fmaf(dz, c.ga[kc], -m1[kk]) - h * m2[kk]));
                }
                XT *const to = addr<XT, V, KIND>(dx, g, g.xs, w, at.p);
                if (CROSS && at.lo > 0) {  // dy of what others own is not here
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (k >= at.lo) to[k] = r.v[k];
                } else if (at.lo < V) {
                    store_vec<XT, V>(to, r);
                }
            }
    });
}

template <int V, int KIND>
__device__ __forceinline__ void take_group_means(const Channels<V, KIND> &c, const float *gm, float *m1, float *m2) {
#pragma unroll
    for (int k = 0; k < c.NG; ++k) {
        m1[k] = gm[2 * c.kg[k]];
        m2[k] = gm[2 * c.kg[k] + 1];
    }
}

template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__global__ __launch_bounds__(1024) void k_norm_bwd_fused(NormGeo g, NormPtrs a) {
    constexpr bool CL = KIND != kPlanar;
    constexpr int NC = thread_channels<V, KIND>(), NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.b;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const red = (float *)smem, *const gm = red + norm_sum_floats(s, CL);
    const Where w = locate<V, KIND>(g, s, b);
    Vec<XT, V> fx[E];
    Vec<YT, V> fd[E];
    load_steps<XT, V, KIND, E>(fx, (const XT *)a.x, g, s, g.xs, w, 0);
    load_dy<YT, V, KIND, CROSS, E>(fd, (const YT *)a.dy, g, w, 0, (YT *)smem);
    Channels<V, KIND> c;
    c.load(g, a, w);
    float s1[NC] = {}, s2[NC] = {}, s3[NC] = {};
    add_sums<XT, YT, V, KIND, E, false>(s1, s2, s3, fx, fd, c, g, w, 0);
    if constexpr (!keeps_derived(V, E, KIND)) {
        forget(fx);
        forget(fd);
    }
    join_sums<V, KIND>(g, a, w, s1, s2, s3, red, gm);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    for (int k = threadIdx.x; k < 2 * s.K; k += blockDim.x)
        a.group[2 * group0 + k] = gm[k] = gm[k] / (float)((double)g.P * g.cpg);
    __syncthreads();
    float m1[NG], m2[NG];
    take_group_means<V, KIND>(c, gm, m1, m2);
    write_dx<XT, YT, V, KIND, CROSS, E>(fx, fd, c, m1, m2, g, w, (XT *)a.dx, 0);
}

template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__global__ __launch_bounds__(kNormSplitThreads) void k_norm_bwd_sums(NormGeo g, NormPtrs a) {
    constexpr bool CL = KIND != kPlanar;
    constexpr int NC = thread_channels<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.b;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const red = (float *)smem, *const gm = red + norm_sum_floats(s, CL);
    const Where w = locate<V, KIND>(g, s, b);
    Vec<XT, V> fx[E];
    Vec<YT, V> fd[E];
    load_steps<XT, V, KIND, E>(fx, (const XT *)a.x, g, s, g.xs, w, 0);
    load_dy<YT, V, KIND, CROSS, E>(fd, (const YT *)a.dy, g, w, 0, (YT *)smem);
    Channels<V, KIND> c;
    c.load(g, a, w);
    float s1[NC] = {}, s2[NC] = {}, s3[NC] = {};
    for (int first = 0;;) {
        add_sums<XT, YT, V, KIND, E, true>(s1, s2, s3, fx, fd, c, g, w, first);
        first += E;
        if (first >= s.steps) break;
        load_steps<XT, V, KIND, E>(fx, (const XT *)a.x, g, s, g.xs, w, first);
        load_dy<YT, V, KIND, CROSS, E>(fd, (const YT *)a.dy, g, w, first, (YT *)smem);
    }
    join_sums<V, KIND>(g, a, w, s1, s2, s3, red, gm);
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    for (int k = threadIdx.x; k < 2 * s.K; k += blockDim.x) {
        const int64_t at = (group0 + k / 2) * (s.nchunk * s.J) + w.chunk * s.J + w.part;
        a.gpart[2 * at + k % 2] = gm[k];
    }
}

template <typename XT, typename YT, int V, int KIND, bool CROSS, int E>
__global__ __launch_bounds__(kNormSplitThreads) void k_norm_bwd_apply(NormGeo g, NormPtrs a) {
    constexpr int NG = group_values<V, KIND>();
    extern __shared__ __align__(16) char smem[];
    const NormShape &s = g.b;
    int b;
    if (!block_number(norm_blocks(g, s), b)) return;
    float *const tot = (float *)smem;
    const Where w = locate<V, KIND>(g, s, b);
    Vec<XT, V> fx[E];
    load_steps<XT, V, KIND, E>(fx, (const XT *)a.x, g, s, g.xs, w, 0);
    Channels<V, KIND> c;
    c.load(g, a, w);
    // the groups' means, a wave joining 4 groups at once, 128 parts at a time
    constexpr int GB = 4, PB = 2;
    const int64_t group0 = (int64_t)w.n * g.G + w.g0;
    const int lane = threadIdx.x & 63, np = s.nchunk * s.J;
    const float m = (float)((double)g.P * g.cpg);
    for (int k0 = (threadIdx.x >> 6) * GB; k0 < s.K; k0 += kNormSplitThreads / 64 * GB) {
        float t1[GB] = {}, t2[GB] = {};
        for (int i0 = 0; i0 < np; i0 += 64 * PB) {
            Vec<float, 2> v[GB][PB];
#pragma unroll
            for (int k = 0; k < GB; ++k)
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    v[k][i] = load_vec<float, 2>(a.gpart + 2 * ((group0 + min(k0 + k, s.K - 1)) * np + min(i0 + i * 64 + lane, np - 1)));
#pragma unroll
            for (int k = 0; k < GB; ++k)
#pragma unroll
                for (int i = 0; i < PB; ++i) {
                    const bool in = i0 + i * 64 + lane < np;
                    t1[k] += in ? v[k][i].v[0] : 0.0f;
                    t2[k] += in ? v[k][i].v[1] : 0.0f;
                }
        }
#pragma unroll
        for (int k = 0; k < GB; ++k) {
            const float m1 = wave_sum(t1[k]) / m, m2 = wave_sum(t2[k]) / m;
            if (lane == 0 && k0 + k < s.K) {
                tot[2 * (k0 + k)] = m1;
                tot[2 * (k0 + k) + 1] = m2;
            }
        }
    }
    __syncthreads();
    if (w.chunk == 0 && w.part == 0)
        for (int k = threadIdx.x; k < 2 * s.K; k += kNormSplitThreads) a.group[2 * group0 + k] = tot[k];
    float m1[NG], m2[NG];
    take_group_means<V, KIND>(c, tot, m1, m2);
    if constexpr (CROSS) __syncthreads();  // the tile takes the means' place
    for (int first = 0;;) {
        Vec<YT, V> fd[E];
        load_dy<YT, V, KIND, CROSS, E>(fd, (const YT *)a.dy, g, w, first, (YT *)smem);
        write_dx<XT, YT, V, KIND, CROSS, E>(fx, fd, c, m1, m2, g, w, (XT *)a.dx, first);
        first += E;
        if (first >= s.steps) break;
        load_steps<XT, V, KIND, E>(fx, (const XT *)a.x, g, s, g.xs, w, first);
    }
}

// dgamma, dbeta: sums of `part` over images and chunks; dshift of image n from
// its own: rstd (gamma S1 - P m1 - m2 S3). 16 channels a block, 16 lanes along
// the rows of `part`; of the rows of blocks, one for each image does its dshift,
// where that is wanted, and the last one, where they are, the parameters' gradients.
__global__ __launch_bounds__(256) void k_norm_params(NormGeo g, NormPtrs a, int ncol, int nblocks) {
    __shared__ float red[2][16][17];
    int b;
    if (!block_number(nblocks, b)) return;
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
    const int n = b / ncol, c = (b - n * ncol) * 16 + tc;
    const bool shift = a.dshift && n < g.N;
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
        const dim3 grid = grid_of(norm_blocks(g, s)), blk(s.threads);
        const size_t red = (size_t)(2 * s.K + 2 * s.slabC + norm_sum_floats(s, KIND != kPlanar)) * 4;
        const size_t tile = CROSS ? tile_lds<YT>(s, KIND != kPlanar) : 0;
        const size_t most = red > tile ? red : tile, means = (size_t)2 * s.K * 4;
        if constexpr (!SPLIT) {
            hipLaunchKernelGGL((k_norm_bwd_fused<XT, YT, V, KIND, CROSS, E>), grid, blk, most, st, g, p);
        } else {
            hipLaunchKernelGGL((k_norm_bwd_sums<XT, YT, V, KIND, CROSS, E>), grid, blk, most, st, g, p);
            hipLaunchKernelGGL((k_norm_bwd_apply<XT, YT, V, KIND, CROSS, E>), grid, blk, means > tile ? means : tile, st, g, p);
        }
    }
};

template <typename XT>
wq8_status norm_backward(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (g.N > 0) {
        if (ydt == WQ8_F32) pick_vector<true, XT, float>(g, RunBackward{g, p, st});
        else pick_vector<true, XT, bf16_t>(g, RunBackward{g, p, st});
    }
    if (p.dgamma || p.dbeta || (p.dshift && g.N > 0)) {
        const int ncol = (g.C + 15) / 16, nblocks = ncol * ((p.dshift ? g.N : 0) + (p.dgamma || p.dbeta ? 1 : 0));
        hipLaunchKernelGGL(k_norm_params, grid_of(nblocks), dim3(256), 0, st, g, p, ncol, nblocks);
    }
    return check_launch("group norm backward");
}

}  // namespace
}  // namespace wq8
