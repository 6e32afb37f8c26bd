// What the group norm's forward and backward kernels share: a block's place in
// the tensors, windows in the other layout, reductions, kernel selection.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "wq8_device.h"
#include "wq8_ops_device.h"

namespace wq8 {
namespace {

enum { kFused = 0, kReduce = 1, kApply = 2 };

// ---------------------------------------------------------- block geometry
struct Where {
    int n, chunk, part;          // part: index along J
    int slab0, cend;             // channels of this block: [slab0, cend)
    int g0;                      // first group
    int p0, pend;                // pixels of this block
    int tp, tc;                  // this thread's place in a window
    int c;                       // its first (NHWC) or only (NCHW) channel
    int nc;                      // its channels that exist (0: it owns nothing)
};

template <int V, bool CL>
__device__ __forceinline__ Where locate(const NormGeo &g, const NormShape &s, int b) {
    Where w;
    const int tid = threadIdx.x;
    w.chunk = b % s.nchunk;
    const int r = b / s.nchunk, slab = r % s.nslab;
    w.n = r / s.nslab;
    if (s.J == 1) {
        w.g0 = slab * s.K;
        w.part = 0;
        w.slab0 = w.g0 * g.cpg;
        w.cend = w.slab0 + s.slabC;
    } else {
        w.g0 = slab / s.J;
        w.part = slab % s.J;
        w.slab0 = w.g0 * g.cpg + w.part * s.slabC;
        w.cend = min(w.slab0 + s.slabC, (w.g0 + 1) * g.cpg);
    }
    w.p0 = w.chunk * s.chunk;
    w.pend = min(w.p0 + s.chunk, g.P);
    if constexpr (CL) {
        w.tc = tid % s.tc;
        w.tp = tid / s.tc;
        w.c = w.slab0 + w.tc * V;
        w.nc = w.tp < s.tp ? min(max(w.cend - w.c, 0), V) : 0;
    } else {
        w.tp = tid % s.tp;
        w.tc = tid / s.tp;
        w.c = w.slab0 + w.tc;
        w.nc = w.c < w.cend;
    }
    return w;
}

// Pixel of step e, and how many of the thread's V elements exist.
template <int V, bool CL>
__device__ __forceinline__ int pixel_of(const NormShape &s, const Where &w, int e) {
    return w.p0 + e * s.window + w.tp * (CL ? 1 : V);
}
template <int V, bool CL>
__device__ __forceinline__ int count_of(const Where &w, int p) {
    if (CL) return p < w.pend ? w.nc : 0;
    return w.nc ? min(max(w.pend - p, 0), V) : 0;
}

// KIND: how a thread's values fall into groups.
//   kPlanar    NCHW: V pixels of one channel
//   kUniform   NHWC: V channels of one group (V divides the group's channels)
//   kStraddle  NHWC: V channels, of any groups; the last thread's may be fewer
enum { kPlanar = 0, kUniform = 1, kStraddle = 2 };

// Values a thread keeps apart in a sum per group.
template <int V, int KIND>
constexpr int group_values() { return KIND == kStraddle ? V : 1; }

// A thread's vector, of which n elements exist: all or none where vectors lie
// within groups.
template <typename T, int V, int KIND>
__device__ __forceinline__ Vec<T, V> load_part(const T *p, int n) {
    if constexpr (KIND == kUniform) {
        Vec<T, V> r = {};
        if (n > 0) r = load_vec<T, V>(p);
        return r;
    } else {
        return load_vec_n<T, V>(p, n);
    }
}
template <typename T, int V, int KIND>
__device__ __forceinline__ void store_part(T *p, const Vec<T, V> &r, int n) {
    if constexpr (KIND == kUniform) {
        if (n > 0) store_vec<T, V>(p, r);
    } else {
        store_vec_n<T, V>(p, r, n);
    }
}

// Makes the compiler forget what it derived from the values: it would keep
// every conversion and sum of one pass over them for the next, several
// registers a value, and spill.
template <typename T, int V, int E>
__device__ __forceinline__ void forget(Vec<T, V> (&f)[E]) {
    constexpr int W = V * sizeof(T) / 4;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        uint32_t u[W];
        __builtin_memcpy(u, &f[e], sizeof u);
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(u[i]));
        __builtin_memcpy(&f[e], u, sizeof u);
    }
}

template <typename T, int V, bool CL>
__device__ __forceinline__ const T *addr(const T *x, const NormGeo &g, int64_t stride, int n, int c,
                                         int p) {
    return CL ? x + ((int64_t)n * g.P + p) * stride + c : x + ((int64_t)n * g.C + c) * g.P + p;
}

// ------------------------------------------------- windows in the other layout
// Threads follow x's layout; tensor `t` has the other one. The tile in LDS
// holds it as t does, [channel][pixel] or [pixel][channel], rows padded by
// two elements to spread the banks.
template <bool CL>
__device__ __forceinline__ int tile_row(const NormShape &s) {
    return (CL ? s.window : s.slabC) + 2;
}

template <typename T, bool CL>
__device__ __forceinline__ void tile_to_global(const T *tile, T *t, const NormGeo &g,
                                               const NormShape &s, const Where &w, int64_t stride,
                                               int p) {
    constexpr int VO = 16 / sizeof(T);
    const int wp = min(s.window, w.pend - p), wc = w.cend - w.slab0, row = tile_row<CL>(s);
    const int inner = CL ? wp : wc, outer = CL ? wc : wp;
    const int nv = (inner + VO - 1) / VO;
    for (int i = threadIdx.x; i < outer * nv; i += blockDim.x) {
        const int o = i / nv, v = (i - o * nv) * VO;
        Vec<T, VO> r;
#pragma unroll
        for (int k = 0; k < VO; ++k) r.v[k] = v + k < inner ? tile[o * row + v + k] : T(0);
        T *dst = CL ? t + ((int64_t)w.n * g.C + w.slab0 + o) * g.P + p + v
                    : t + ((int64_t)w.n * g.P + p + o) * stride + w.slab0 + v;
        store_vec_n<T, VO>(dst, r, inner - v);
    }
}

template <typename T, bool CL>
__device__ __forceinline__ void global_to_tile(T *tile, const T *t, const NormGeo &g,
                                               const NormShape &s, const Where &w, int64_t stride,
                                               int p) {
    constexpr int VO = 16 / sizeof(T);
    const int wp = min(s.window, w.pend - p), wc = w.cend - w.slab0, row = tile_row<CL>(s);
    const int inner = CL ? wp : wc, outer = CL ? wc : wp;
    const int nv = (inner + VO - 1) / VO;
    for (int i = threadIdx.x; i < outer * nv; i += blockDim.x) {
        const int o = i / nv, v = (i - o * nv) * VO;
        const T *src = CL ? t + ((int64_t)w.n * g.C + w.slab0 + o) * g.P + p + v
                          : t + ((int64_t)w.n * g.P + p + o) * stride + w.slab0 + v;
        const Vec<T, VO> r = load_vec_n<T, VO>(src, inner - v);
#pragma unroll
        for (int k = 0; k < VO; ++k)
            if (v + k < inner) tile[o * row + v + k] = r.v[k];
    }
}

// The tile's place of element k of this thread.
template <bool CL, int V>
__device__ __forceinline__ int tile_at(const NormShape &s, const Where &w, int k) {
    return CL ? (w.tc * V + k) * tile_row<CL>(s) + w.tp
              : (w.tp * V + k) * tile_row<CL>(s) + w.tc;
}

// ------------------------------------------------------------- reductions
// Sum of each channel over the block's pixels: thread values v[V] (NHWC: V
// channels; NCHW: v[0] of one channel, zero where the thread owns none) ->
// out[slabC] in LDS. `lds` holds threads * V floats (NHWC) and then
// max(threads, slabC).
template <int V, bool CL>
__device__ __forceinline__ void channel_sum(const float (&v)[CL ? V : 1], const NormShape &s,
                                            const Where &w, float *lds, float *out) {
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, nw = T >> 6;
    float *const lds2 = lds + (CL ? T * V : 0);
    int Q;
    if constexpr (CL) {
        const int row = s.tc * V;
        if (w.tp < s.tp)
#pragma unroll
            for (int k = 0; k < V; ++k) lds[w.tp * row + w.tc * V + k] = k < w.nc ? v[k] : 0.0f;
        __syncthreads();
        Q = max(1, min(T / s.slabC, s.tp));
        for (int i = tid; i < s.slabC * Q; i += T) {
            const int q = i / s.slabC, c = i - q * s.slabC;
            float t = 0.0f;
            for (int r = q; r < s.tp; r += Q) t += lds[r * row + c];
            lds2[c * Q + q] = t;
        }
    } else {
        Q = s.tp;
        if (w.tc < s.slabC) lds2[w.tc * Q + w.tp] = v[0];
    }
    __syncthreads();
    if (Q <= 16) {
        for (int c = tid; c < s.slabC; c += T) {
            float t = 0.0f;
            for (int q = 0; q < Q; ++q) t += lds2[c * Q + q];
            out[c] = t;
        }
    } else {
        for (int c = wave; c < s.slabC; c += nw) {
            float t = 0.0f;
            for (int q = lane; q < Q; q += 64) t += lds2[c * Q + q];
            t = wave_sum(t);
            if (lane == 0) out[c] = t;
        }
    }
    __syncthreads();
}

// Totals of the block's K groups in LDS, from per-channel sums weighted by
// gamma (or 1): a wave per group.
template <typename F>
__device__ __forceinline__ void groups_of_channels(const NormGeo &g, const NormShape &s, const Where &w, F weighted,
                                                   float *tot, int stride) {
    const int lane = threadIdx.x & 63, nc = s.J == 1 ? g.cpg : w.cend - w.slab0;
    for (int k = threadIdx.x >> 6; k < s.K; k += blockDim.x >> 6) {
        float t = 0.0f;
        for (int i = lane; i < nc; i += 64) t += weighted(k * g.cpg + i);
        t = wave_sum(t);
        if (lane == 0) tot[k * stride] = t;
    }
}

// Sum over the block of each of its K groups -> tot[K] in LDS. Ends with a
// barrier; `lds` as for channel_sum, then slabC floats.
template <int V, int KIND>
__device__ __forceinline__ void group_sum(const float (&v)[group_values<V, KIND>()], const NormGeo &g,
                                          const NormShape &s, const Where &w, float *lds, float *tot) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    if (s.K == 1) {
        float u = 0.0f;
#pragma unroll
        for (int k = 0; k < group_values<V, KIND>(); ++k)
            if (k < w.nc) u += v[k];
        u = wave_sum(u);
        if (lane == 0) lds[wave] = u;
        __syncthreads();
        if (wave == 0) {
            u = wave_sum(lane < nw ? lds[lane] : 0.0f);
            if (lane == 0) tot[0] = u;
        }
    } else if constexpr (KIND == kStraddle) {
        float *chan = lds + blockDim.x * V + max((int)blockDim.x, s.slabC);
        channel_sum<V, true>(v, s, w, lds, chan);
        groups_of_channels(g, s, w, [&](int c) { return chan[c]; }, tot, 1);
    } else {
        lds[tid] = w.nc ? v[0] : 0.0f;
        __syncthreads();
        constexpr bool CL = KIND == kUniform;
        const int per = CL ? g.cpg / V : g.cpg * s.tp;  // a row of one group's threads
        const int rows = CL ? s.tp : 1;
        for (int k = wave; k < s.K; k += nw) {
            float t = 0.0f;
            for (int i = lane; i < per * rows; i += 64) {
                const int r = i / per;
                t += lds[r * s.tc + k * per + i - r * per];
            }
            t = wave_sum(t);
            if (lane == 0) tot[k] = t;
        }
    }
    __syncthreads();
}

// Group, counted from the block's first, of the thread's k-th value.
template <int V, int KIND>
__device__ __forceinline__ int group_of(const NormGeo &g, const NormShape &s, const Where &w, int k) {
    if (s.J > 1) return 0;
    const int c = w.c - w.slab0 + (KIND == kStraddle ? k : 0);
    return min(c / g.cpg, s.K - 1);
}

// Values of a per-channel array for this thread's channels (1 for NCHW).
template <int V, bool CL>
__device__ __forceinline__ void per_channel(float (&r)[CL ? V : 1], const float *a, int64_t at, int nc,
                                            float none) {
#pragma unroll
    for (int k = 0; k < (CL ? V : 1); ++k) r[k] = a && k < nc ? a[at + k] : none;
}

// -------------------------------------------------------------- launching
// Floats of LDS that group_sum or channel_sum takes, without their results.
inline int sum_floats(const NormShape &s, int kind) {
    return (kind == kPlanar ? 0 : s.threads * s.V) + (s.threads > s.slabC ? s.threads : s.slabC);
}

template <typename T>
size_t tile_lds(const NormShape &s, bool cl) {
    return (size_t)(cl ? s.tc * s.V : s.window) * ((cl ? s.window : s.slabC) + 2) * sizeof(T);
}

// Calls run<XT, YT, V, KIND, CROSS, SPLIT, E>() for the plan's types, layouts
// and shape.
template <bool BWD, typename XT, typename YT, int V, int KIND, typename R>
void pick_steps(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    const auto go = [&](auto split, auto e) {
        constexpr bool S = decltype(split)::value;
        constexpr int E = decltype(e)::value;
        if (g.x_nhwc != g.y_nhwc) run.template operator()<XT, YT, V, KIND, true, S, E>();
        else run.template operator()<XT, YT, V, KIND, false, S, E>();
    };
    if (s.split) go(std::true_type{}, std::integral_constant<int, norm_split_steps(BWD)>{});
    else if (s.steps <= kNormE) go(std::false_type{}, std::integral_constant<int, kNormE>{});
    else go(std::false_type{}, std::integral_constant<int, norm_max_steps(BWD)>{});
}

template <bool BWD, typename XT, typename YT, typename R>
void pick_vector(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    constexpr int VM = norm_max_vec(sizeof(XT), sizeof(YT));
    if (!g.x_nhwc) return pick_steps<BWD, XT, YT, VM, kPlanar>(g, run);
    if (g.cpg % s.V != 0) return pick_steps<BWD, XT, YT, VM, kStraddle>(g, run);
    if constexpr (VM == 8)
        if (s.V == 8) return pick_steps<BWD, XT, YT, 8, kUniform>(g, run);
    pick_steps<BWD, XT, YT, 4, kUniform>(g, run);
}

template <bool BWD, typename R>
void pick_kernel(const NormGeo &g, wq8_dtype xdt, wq8_dtype ydt, const R &run) {
    if (xdt == WQ8_F32) {
        if (ydt == WQ8_F32) pick_vector<BWD, float, float>(g, run);
        else pick_vector<BWD, float, bf16_t>(g, run);
    } else {
        if (ydt == WQ8_F32) pick_vector<BWD, bf16_t, float>(g, run);
        else pick_vector<BWD, bf16_t, bf16_t>(g, run);
    }
}

}  // namespace
}  // namespace wq8
