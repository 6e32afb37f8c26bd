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
// KIND: how a thread's values fall into channels and groups.
//   kPlanar    NCHW: V pixels of one channel
//   kUniform   NHWC: V channels of one group (V divides the group's channels)
//   kStraddle  NHWC: V channels, of any groups
// A vector that would pass the end of its row starts earlier instead, so that
// every load is a whole vector inside the tensor: its first `lo` values belong
// to another thread. They are left out of the sums; stored, they are the
// values that the other thread stores. lo = V: the thread owns nothing there,
// and what it loads is any valid vector.
enum { kPlanar = 0, kUniform = 1, kStraddle = 2 };

// Channels of a thread, and values it keeps apart in a sum per group.
template <int V, int KIND>
constexpr int thread_channels() { return KIND == kPlanar ? 1 : V; }
template <int V, int KIND>
constexpr int group_values() { return KIND == kStraddle ? V : 1; }

struct Where {
    int n, chunk, part;          // part: index along J
    int slab0, cend;             // channels of this block: [slab0, cend)
    int g0;                      // first group
    int p0, pend;                // pixels of this block
    int tp, tc;                  // this thread's place in a window
    int c;                       // its first (NHWC) or only (NCHW) channel
    int lo;                      // its channels that others own
};

__host__ __device__ inline int norm_blocks(const NormGeo &g, const NormShape &s) { return g.N * s.nslab * s.nchunk; }

template <int V, int KIND>
__device__ __forceinline__ Where locate(const NormGeo &g, const NormShape &s, int block) {
    Where w;
    const int b = xcd_block(block, norm_blocks(g, s)), tid = threadIdx.x;
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
    if constexpr (KIND != kPlanar) {
        w.tc = tid % s.tc;
        w.tp = tid / s.tc;
        const int c = w.slab0 + w.tc * V;
        w.c = min(c, w.cend - V);
        w.lo = w.tp < s.tp ? min(c - w.c, V) : V;
    } else {
        w.tp = tid % s.tp;
        w.tc = tid / s.tp;
        const int c = w.slab0 + w.tc;
        w.c = min(c, w.cend - 1);
        w.lo = c == w.c ? 0 : V;
    }
    return w;
}

// First pixel of the thread's vector in step e, and its values that others own.
struct Step {
    int p, lo;
};
template <int V, int KIND>
__device__ __forceinline__ Step step_of(const NormShape &s, const Where &w, int e) {
    if constexpr (KIND != kPlanar) {
        const int p = w.p0 + e * s.window + w.tp;
        return {min(p, w.pend - 1), p < w.pend ? w.lo : V};
    } else {
        const int p = w.p0 + e * s.window + w.tp * V, q = min(p, w.pend - V);
        return {q, w.lo ? V : min(p - q, V)};
    }
}

template <typename T, int V, int KIND>
__device__ __forceinline__ T *addr(T *x, const NormGeo &g, int64_t stride, const Where &w, int p) {
    return KIND != kPlanar ? x + ((int64_t)w.n * g.P + p) * stride + w.c : x + ((int64_t)w.n * g.C + w.c) * g.P + p;
}

// The thread's vectors of E steps from step `first`. Steps past the block's last
// one load its last vector again: a load under a condition would be waited for
// before the next one is sent.
template <typename T, int V, int KIND, int E>
__device__ __forceinline__ void load_steps(Vec<T, V> (&f)[E], const T *x, const NormGeo &g, const NormShape &s, int64_t stride,
                                           const Where &w, int first) {
#pragma unroll
    for (int e = 0; e < E; ++e)
        f[e] = load_vec<T, V>(addr<const T, V, KIND>(x, g, stride, w, step_of<V, KIND>(s, w, first + e).p));
}

// f(e, k, ok) for the values of E steps from step `first`; ok: the value is one
// of the block's, and in NCHW no other thread's vector has it. What a thread or
// a channel that owns nothing has summed, drop_unowned() clears. BATCH: where
// the steps end before the block's pixels do, ok is the constant true (two
// copies of the code, too many registers where the values are held for more).
template <int V, int KIND, int E, bool BATCH, typename F>
__device__ __forceinline__ void for_values(const NormShape &s, const Where &w, int first, F f) {
    if (BATCH && w.p0 + (first + E) * s.window <= w.pend) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int k = 0; k < V; ++k) f(e, k, std::true_type{});
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int p = w.p0 + (first + e) * s.window + w.tp * (KIND == kPlanar ? V : 1);
            const bool in = p < w.pend;
            const int lo = KIND == kPlanar ? step_of<V, KIND>(s, w, first + e).lo : 0;
#pragma unroll
            for (int k = 0; k < V; ++k) f(e, k, KIND == kPlanar ? k >= lo : in);
        }
    }
}

// Sums of what the thread does not own: nothing.
template <int V, int KIND, int N>
__device__ __forceinline__ void drop_unowned(const Where &w, float (&sum)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (N == 1 ? w.lo == V || (KIND == kPlanar && w.lo) : k < w.lo) sum[k] = 0.0f;
}

// Whether there are registers to keep what one pass over the values derived
// from them for the next one.
constexpr bool keeps_derived(int V, int E, int kind) { return V * E <= (kind == kStraddle ? 16 : 32); }

// Makes the compiler forget what it derived from the values: it would keep
// every conversion and sum, several registers a value, and spill.
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

// ------------------------------------------------- windows in the other layout
// Threads follow x's layout; tensor `t` has the other one. The tile in LDS
// holds `tsteps` windows of it as t does, [channel][pixel] or [pixel][channel],
// rows padded by two elements to spread the banks.
template <bool CL>
__device__ __forceinline__ int tile_row(const NormShape &s) {
    return (CL ? s.tsteps * s.window : s.slabC) + 2;
}

// Rows and their length of the tile whose first pixel is p.
template <bool CL>
__device__ __forceinline__ void tile_extent(const NormShape &s, const Where &w, int p, int &outer, int &inner) {
    const int wp = min(s.tsteps * s.window, w.pend - p), wc = w.cend - w.slab0;
    inner = CL ? wp : wc;
    outer = CL ? wc : wp;
}

template <typename T, bool CL>
__device__ __forceinline__ T *tile_addr(T *t, const NormGeo &g, const Where &w, int64_t stride, int p, int row, int at) {
    return CL ? t + ((int64_t)w.n * g.C + w.slab0 + row) * g.P + p + at
              : t + ((int64_t)w.n * g.P + p + row) * stride + w.slab0 + at;
}

// The tile's vectors are shared out over the block, 4 to a thread at a time with
// their loads in flight. A vector that would pass the end of its row starts
// earlier and carries some values twice.
constexpr int kTileBatch = 4;

template <typename T, bool CL, typename F>
__device__ __forceinline__ void for_tile(const NormShape &s, const Where &w, int p, F f) {
    constexpr int VO = 16 / sizeof(T);
    int outer, inner;
    tile_extent<CL>(s, w, p, outer, inner);
    const int nv = (inner + VO - 1) / VO, total = outer * nv;
    for (int i0 = threadIdx.x; i0 < total; i0 += kTileBatch * blockDim.x) {
        int row[kTileBatch], at[kTileBatch];
#pragma unroll
        for (int j = 0; j < kTileBatch; ++j) {
            const int i = min(i0 + j * (int)blockDim.x, total - 1);
            row[j] = i / nv;
            at[j] = min((i - row[j] * nv) * VO, max(inner - VO, 0));
        }
        f(row, at, inner);
    }
}

template <typename T, bool CL>
__device__ __forceinline__ void tile_to_global(const T *tile, T *t, const NormGeo &g, const NormShape &s, const Where &w,
                                               int64_t stride, int p) {
    constexpr int VO = 16 / sizeof(T);
    const int trow = tile_row<CL>(s);
    for_tile<T, CL>(s, w, p, [&](const int *row, const int *at, int inner) {
#pragma unroll
        for (int j = 0; j < kTileBatch; ++j) {
            Vec<T, VO> r;
#pragma unroll
            for (int k = 0; k < VO; ++k) r.v[k] = tile[row[j] * trow + at[j] + (inner < VO ? min(k, inner - 1) : k)];
            T *const to = tile_addr<T, CL>(t, g, w, stride, p, row[j], at[j]);
            if (inner >= VO) store_vec<T, VO>(to, r);
            else store_vec_n<T, VO>(to, r, inner);
        }
    });
}

template <typename T, bool CL>
__device__ __forceinline__ void global_to_tile(T *tile, const T *t, const NormGeo &g, const NormShape &s, const Where &w,
                                               int64_t stride, int p) {
    constexpr int VO = 16 / sizeof(T);
    const int trow = tile_row<CL>(s);
    for_tile<T, CL>(s, w, p, [&](const int *row, const int *at, int inner) {
        Vec<T, VO> r[kTileBatch];
        if (inner >= VO) {
#pragma unroll
            for (int j = 0; j < kTileBatch; ++j)
                r[j] = load_vec<T, VO>(tile_addr<const T, CL>(t, g, w, stride, p, row[j], at[j]));
        } else {
#pragma unroll
            for (int j = 0; j < kTileBatch; ++j)
                r[j] = load_vec_n<T, VO>(tile_addr<const T, CL>(t, g, w, stride, p, row[j], at[j]), inner);
        }
#pragma unroll
        for (int j = 0; j < kTileBatch; ++j)
#pragma unroll
            for (int k = 0; k < VO; ++k)
                if (k < inner) tile[row[j] * trow + at[j] + k] = r[j].v[k];
    });
}

// The tile's place of value k of a vector that starts at pixel p; the tile
// starts at pixel p0.
template <int V, int KIND>
__device__ __forceinline__ int tile_at(const NormShape &s, const Where &w, int p0, int p, int k) {
    return KIND != kPlanar ? (w.c - w.slab0 + k) * tile_row<true>(s) + p - p0
                           : (p - p0 + k) * tile_row<false>(s) + w.c - w.slab0;
}

// ------------------------------------------------------------- reductions
// Sum of each channel over the block's pixels: thread values v[V] (NHWC: V
// channels; NCHW: v[0] of one channel; zero where the thread owns none) ->
// out[slabC] in LDS. `lds` holds threads * V floats (NHWC) and then
// max(threads, slabC).
template <int V, bool CL>
__device__ __forceinline__ void channel_sum(const float (&v)[CL ? V : 1], const NormShape &s,
                                            const Where &w, float *lds, float *out) {
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, nw = T >> 6;
    float *const lds2 = lds + (CL ? T * V : 0);
    int Q;
    if constexpr (CL) {
        const int nc = w.cend - w.slab0, nv = (nc + V - 1) / V, row = s.tc * V, last = (nv - 1) * V, shift = nv * V - nc;
        if (w.tp < s.tp) {
            if constexpr (V == 1) {
                lds[w.tp * row + w.tc] = v[0];
            } else {
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    *(float4 *)(lds + w.tp * row + w.tc * V + k) = float4{v[k], v[k + 1], v[k + 2], v[k + 3]};
            }
        }
        __syncthreads();
        Q = max(1, min(T / s.slabC, s.tp));
        for (int i = tid; i < s.slabC * Q; i += T) {
            const int q = i / s.slabC, c = i - q * s.slabC;
            if (c >= nc) continue;
            float t = 0.0f;
            // the last column's vector starts `shift` channels early
            for (int r = q; r < s.tp; r += Q) t += lds[r * row + c + (c >= last ? shift : 0)];
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

// Sum over the block of each of its K groups -> tot[K] in LDS, from values that
// are zero where a thread owns none. Ends with a barrier; `lds` as for channel_sum.
template <int V, int KIND>
__device__ __forceinline__ void group_sum(const float (&v)[group_values<V, KIND>()], const NormGeo &g,
                                          const NormShape &s, const Where &w, float *lds, float *tot) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    if (s.K == 1) {
        float u = 0.0f;
#pragma unroll
        for (int k = 0; k < group_values<V, KIND>(); ++k)
            u += v[k];
        u = wave_sum(u);
        if (lane == 0) lds[wave] = u;
        __syncthreads();
        if (wave == 0) {
            u = wave_sum(lane < nw ? lds[lane] : 0.0f);
            if (lane == 0) tot[0] = u;
        }
    } else if constexpr (KIND == kStraddle) {
        // each thread's values by group, the j-th of its groups in its slot j
        const auto start = [&](int col) { return min(col * V, s.slabC - V); };
        const int S = min((V - 1) / g.cpg + 2, V), c0 = start(w.tc), first = c0 / g.cpg;
        for (int j = 0; j < S; ++j) {
            const int a = (first + j) * g.cpg - c0;  // values [a, a + cpg) are of the group
            float u = 0.0f;
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k >= a && k < a + g.cpg) u += v[k];
            lds[tid * S + j] = u;
        }
        __syncthreads();
        for (int k = wave; k < s.K; k += nw) {
            // columns that own values of group k
            const int a = k * g.cpg / V, n = ((k + 1) * g.cpg - 1) / V - a + 1;
            float t = 0.0f;
            for (int i = lane; i < n * s.tp; i += 64) {
                const int r = i / n, col = a + i - r * n;
                t += lds[(r * s.tc + col) * S + k - start(col) / g.cpg];
            }
            t = wave_sum(t);
            if (lane == 0) tot[k] = t;
        }
    } else {
        lds[tid] = v[0];
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

// Groups, counted from the block's first, of the thread's channels.
template <int V, int KIND>
__device__ __forceinline__ void groups_of(int *kg, const NormGeo &g, const NormShape &s, const Where &w) {
    const int c = w.c - w.slab0;
    int k = s.J > 1 ? 0 : c / g.cpg, left = s.J > 1 ? V + 1 : g.cpg - (c - k * g.cpg);
#pragma unroll
    for (int i = 0; i < thread_channels<V, KIND>(); ++i) {
        kg[i] = k;
        if (KIND == kStraddle && --left == 0) {
            ++k;
            left = g.cpg;
        }
    }
}

// Values of a per-channel array for this thread's channels; ones or zeros for
// an array that is not given, from memory as well, so that no load waits for
// another one's condition.
static __device__ const float kOnes[8] = {1, 1, 1, 1, 1, 1, 1, 1};
static __device__ const float kZeros[8] = {};

template <int V, int KIND>
__device__ __forceinline__ void per_channel(float *r, const float *a, int64_t at, const float *none) {
    constexpr int NC = thread_channels<V, KIND>();
    const Vec<float, NC> v = load_vec<float, NC>(a ? a + at : none);
#pragma unroll
    for (int k = 0; k < NC; ++k) r[k] = v.v[k];
}

// -------------------------------------------------------------- launching
template <typename T>
size_t tile_lds(const NormShape &s, bool cl) {
    const int window = s.tsteps * s.window;
    return (size_t)(cl ? s.slabC : window) * ((cl ? window : s.slabC) + 2) * sizeof(T);
}

// Calls run<XT, YT, V, KIND, CROSS, SPLIT, E>() for the plan's types, layouts
// and shape.
template <bool BWD, typename XT, typename YT, int V, int KIND, typename R>
void pick_steps(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    const auto go = [&](auto cross) {
        constexpr bool X = decltype(cross)::value;
        // single pixels are taken one by one of images that hold no vector: few steps
        constexpr bool FEW = KIND == kPlanar && V == 1 && norm_max_vec(sizeof(XT), sizeof(YT), BWD) <= kNormE;
        if (s.split) run.template operator()<XT, YT, V, KIND, X, true, kNormE>();
        else if (FEW || s.steps <= kNormE) run.template operator()<XT, YT, V, KIND, X, false, kNormE>();
        else run.template operator()<XT, YT, V, KIND, X, false, FEW ? kNormE : norm_max_steps(BWD, KIND == kStraddle, X)>();
    };
    if (g.x_nhwc != g.y_nhwc) go(std::true_type{});
    else go(std::false_type{});
}

template <bool BWD, typename XT, typename YT, typename R>
void pick_vector(const NormGeo &g, const R &run) {
    const NormShape &s = BWD ? g.b : g.f;
    constexpr int VM = norm_max_vec(sizeof(XT), sizeof(YT), BWD);
    if (!g.x_nhwc) return s.V == 1 ? pick_steps<BWD, XT, YT, 1, kPlanar>(g, run) : pick_steps<BWD, XT, YT, VM, kPlanar>(g, run);
    if (s.V == 1) return pick_steps<BWD, XT, YT, 1, kUniform>(g, run);
    if (g.cpg % s.V != 0) return pick_steps<BWD, XT, YT, VM, kStraddle>(g, run);
    if constexpr (VM == 8)
        if (s.V == 8) return pick_steps<BWD, XT, YT, 8, kUniform>(g, run);
    pick_steps<BWD, XT, YT, 4, kUniform>(g, run);
}

}  // namespace
}  // namespace wq8
