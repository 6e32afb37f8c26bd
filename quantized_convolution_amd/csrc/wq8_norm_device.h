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
    int n, chunk, slab, part;    // part: index along J
    int slab0, cend;             // channels of this block: [slab0, cend)
    int g0;                      // first group
    int p0, pend;                // pixels of this block
    int tc, tp;                  // this thread's place in a window
    int c;                       // its first (NHWC) or only (NCHW) channel
    bool on;                     // it owns elements
    int kg;                      // its group, counted from g0
};

template <int V, bool CL>
__device__ __forceinline__ Where locate(const NormGeo &g, const NormShape &s) {
    Where w;
    const int b = xcd_block(blockIdx.x, gridDim.x), tid = threadIdx.x;
    w.chunk = b % s.nchunk;
    const int r = b / s.nchunk;
    w.slab = r % s.nslab;
    w.n = r / s.nslab;
    if (s.J == 1) {
        w.g0 = w.slab * s.K;
        w.part = 0;
        w.slab0 = w.g0 * g.cpg;
        w.cend = w.slab0 + s.slabC;
    } else {
        w.g0 = w.slab / s.J;
        w.part = w.slab % s.J;
        w.slab0 = w.g0 * g.cpg + w.part * s.slabC;
        w.cend = min(w.slab0 + s.slabC, (w.g0 + 1) * g.cpg);
    }
    w.p0 = w.chunk * s.chunk;
    w.pend = min(w.p0 + s.chunk, g.P);
    if constexpr (CL) {
        w.tc = tid % s.tc;
        w.tp = tid / s.tc;
        w.c = w.slab0 + w.tc * V;
        w.on = w.tp < s.tp && w.c < w.cend;
    } else {
        w.tp = tid % s.tp;
        w.tc = tid / s.tp;
        w.c = w.slab0 + w.tc;
        w.on = w.c < w.cend;
    }
    w.kg = w.on && s.J == 1 ? (w.c - w.slab0) / g.cpg : 0;
    return w;
}

// Pixel of step e, and how many of the thread's V elements exist (NHWC: V or
// none).
template <int V, bool CL>
__device__ __forceinline__ int pixel_of(const NormShape &s, const Where &w, int e) {
    return CL ? w.p0 + e * s.window + w.tp : w.p0 + e * s.window + w.tp * V;
}
template <int V, bool CL>
__device__ __forceinline__ int count_of(const Where &w, int p) {
    if (!w.on) return 0;
    if (CL) return p < w.pend ? V : 0;
    return min(max(w.pend - p, 0), V);
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
        const int o = i / nv, v = (i % nv) * VO;
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
        const int o = i / nv, v = (i % nv) * VO;
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
// Sum over the threads of each of the block's K groups; every thread gets its
// own group's. `lds` holds blockDim.x + K floats. Two barriers; the caller
// places one before it writes the same LDS again.
template <int V, bool CL>
__device__ __forceinline__ float group_sum(float v, const NormGeo &g, const NormShape &s,
                                           const Where &w, float *lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    if (s.K == 1) {
        v = wave_sum(w.on ? v : 0.0f);
        if (lane == 0) lds[wave] = v;
        __syncthreads();
        float t = 0.0f;
        for (int i = 0; i < nw; ++i) t += lds[i];
        __syncthreads();
        return t;
    }
    float *tot = lds + blockDim.x;
    lds[tid] = w.on ? v : 0.0f;
    __syncthreads();
    const int per = CL ? g.cpg / V : g.cpg * s.tp;  // a row of one group's threads
    const int rows = CL ? s.tp : 1;
    for (int k = wave; k < s.K; k += nw) {
        float t = 0.0f;
        for (int i = lane; i < per * rows; i += 64) t += lds[(i / per) * s.tc * (CL ? 1 : 0) + k * per + i % per];
        t = wave_sum(t);
        if (lane == 0) tot[k] = t;
    }
    __syncthreads();
    const float t = tot[w.kg];
    __syncthreads();
    return t;
}

// Sum of each channel over the block's pixels: thread values v[V] (NHWC: V
// channels; NCHW: v[0] of one channel) -> out[slabC] in LDS. `lds` holds
// threads * V floats for the rows and `lds2` max(threads, slabC) + slabC.
template <int V, bool CL>
__device__ __forceinline__ void channel_sum(const float (&v)[CL ? V : 1], const NormShape &s,
                                            const Where &w, float *lds, float *lds2, float *out) {
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, nw = T >> 6;
    int Q;
    if constexpr (CL) {
        if (w.tp < s.tp)
#pragma unroll
            for (int k = 0; k < V; ++k) lds[w.tp * s.slabC + w.tc * V + k] = w.on ? v[k] : 0.0f;
        __syncthreads();
        Q = max(1, min(T / s.slabC, s.tp));
        for (int i = tid; i < s.slabC * Q; i += T) {
            const int c = i % s.slabC, q = i / s.slabC;
            float t = 0.0f;
            for (int r = q; r < s.tp; r += Q) t += lds[r * s.slabC + c];
            lds2[c * Q + q] = t;
        }
    } else {
        Q = s.tp;
        if (w.tc < s.slabC) lds2[w.tc * Q + w.tp] = w.on ? v[0] : 0.0f;
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

// Values of a per-channel array for this thread's channels (1 for NCHW).
template <int V, bool CL>
__device__ __forceinline__ void per_channel(float (&r)[CL ? V : 1], const float *a, int64_t at, bool on,
                                            float none) {
#pragma unroll
    for (int k = 0; k < (CL ? V : 1); ++k) r[k] = a && on ? a[at + k] : none;
}

// -------------------------------------------------------------- launching
size_t reduce_lds(const NormShape &s, bool cl, bool backward) {
    if (!backward) return (size_t)(s.threads + s.K) * 4;
    const int rows = cl ? s.threads * s.V : 0;
    return (size_t)(rows + (s.threads > s.slabC ? s.threads : s.slabC) + 3 * s.slabC + 2 * s.K) * 4;
}

template <typename T>
size_t tile_lds(const NormShape &s, bool cl) {
    return (size_t)(cl ? s.slabC : s.window) * ((cl ? s.window : s.slabC) + 2) * sizeof(T);
}

// Calls run<XT, YT, V, CL, CROSS, E>() for the plan's types, layouts and shape.
template <bool BWD, typename XT, typename YT, int V, bool CL, typename R>
void pick_steps(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    using E0 = std::integral_constant<int, kNormE>;
    using E1 = std::integral_constant<int, norm_max_steps(V, BWD)>;
    const auto go = [&](auto cross, auto e) {
        run.template operator()<XT, YT, V, CL, decltype(cross)::value, decltype(e)::value>();
    };
    if (g.x_nhwc != g.y_nhwc) s.E == kNormE ? go(std::true_type{}, E0{}) : go(std::true_type{}, E1{});
    else s.E == kNormE ? go(std::false_type{}, E0{}) : go(std::false_type{}, E1{});
}

template <bool BWD, typename XT, typename YT, typename R>
void pick_vector(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    constexpr int VM = norm_max_vec(sizeof(XT), sizeof(YT));
    if (!g.x_nhwc) return pick_steps<BWD, XT, YT, VM, false>(g, run);
    if constexpr (VM == 8)
        if (s.V == 8) return pick_steps<BWD, XT, YT, 8, true>(g, run);
    if (s.V == 4) return pick_steps<BWD, XT, YT, 4, true>(g, run);
    if (s.V == 2) return pick_steps<BWD, XT, YT, 2, true>(g, run);
    pick_steps<BWD, XT, YT, 1, true>(g, run);
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
