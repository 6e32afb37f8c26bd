// Root-mean-square norm with the residual's addition, and the packing of rows
// to codes, which is the same pass without the norm.
//
// A row is held in registers, as it lies in memory, between its one read and
// its one write: by a wave up to 4096 columns, by a block up to 32768. Longer
// ones are read twice. Memory bounds it: some 10 operations a value. 16384 x 2560
// bf16 with a residual, the stream and codes out take 60 us, 294 MB at 4.9 TB/s, a
// wave a row; with every load bounded by the last column 123 us. 8192 x 5120 bf16
// packed takes 26 us (4.8 TB/s) in blocks of 256, one row of 1280 3.1 us.
// The codes are those of h gamma, before the norm's factor: that is the same
// for the whole row and only enters its scale, so codes need no second
// rounding, and do not hang on the last bit of a sum.
#pragma once

#include "wq8_rows.h"

namespace wq8 {
namespace {

__device__ __forceinline__ float rms_factor(float sum, const RowsGeo &g) {
    return 1.0f / __builtin_sqrtf(sum / (float)g.C + g.eps);
}

template <typename XT>
__device__ __forceinline__ Vec<XT, kV> add_rounded(const Vec<XT, kV> &x, const Vec<XT, kV> &r) {
    Vec<XT, kV> h;
#pragma unroll
    for (int k = 0; k < kV; ++k) h.v[k] = from_f32<XT>(to_f32(x.v[k]) + to_f32(r.v[k]));
    return h;
}

// What a thread adds to its row's sum of squares and largest |h gamma|.
template <typename XT, bool NORM>
__device__ __forceinline__ void take(const Vec<XT, kV> &h, const Vec<float, kV> &gm, float &sum, float &most) {
#pragma unroll
    for (int k = 0; k < kV; ++k) {
        const float v = to_f32(h.v[k]);
        if constexpr (NORM) {
            sum = fmaf(v, v, sum);
            most = larger(most, v * gm.v[k]);
        } else {
            most = larger(most, v);
        }
    }
}

template <typename XT, typename YT>
__device__ __forceinline__ Vec<YT, kV> normed(const Vec<XT, kV> &h, const Vec<float, kV> &gm, float rstd) {
    Vec<YT, kV> y;
#pragma unroll
    for (int k = 0; k < kV; ++k) y.v[k] = from_f32<YT>(to_f32(h.v[k]) * rstd * gm.v[k]);
    return y;
}

template <typename XT, bool NORM>
__device__ __forceinline__ uint64_t coded(const Vec<XT, kV> &h, const Vec<float, kV> &gm, const Coder &code) {
    float t[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) t[k] = NORM ? to_f32(h.v[k]) * gm.v[k] : to_f32(h.v[k]);
    return code.pack(t);
}

template <bool NORM>
__device__ __forceinline__ void give_row(const RmsPtrs &a, int64_t row, float rstd, const Coder &code) {
    if (!NORM || a.codes) a.scales[row] = NORM ? code.scale * rstd : code.scale;
    if (NORM && a.rstd) a.rstd[row] = rstd;
}

template <typename XT, typename YT, int L, int U, bool NORM>
__global__ __launch_bounds__(L < 256 ? 256 : L) void k_row(RowsGeo g, RmsPtrs a, int blocks) {
    constexpr int PER = L < 256 ? 256 / L : 1;
    __shared__ float red[L > 64 ? 2 * L / 64 : 1];
    int b;
    if (!block_number(blocks, b)) return;
    const int64_t row = (int64_t)b * PER + (L < 256 ? threadIdx.x / L : 0);
    if (row >= g.rows) return;  // a whole wave, which meets no barrier
    const int t = threadIdx.x % L;
    Vec<XT, kV> h[U];
    Vec<float, kV> gm[U];
    load_row<XT, L, U>(h, (const XT *)a.x + row * g.xs, t, g.C);
    if constexpr (NORM) {
        load_gamma<L, U>(gm, a.gamma, t, g.C);
        if (a.residual) {  // the last loads: all are on their way before one is waited for
            Vec<XT, kV> o[U];
            load_row<XT, L, U>(o, (const XT *)a.residual + row * g.xs, t, g.C);
#pragma unroll
            for (int s = 0; s < U; ++s) h[s] = add_rounded(h[s], o[s]);
        }
        if (a.h)
#pragma unroll
            for (int s = 0; s < U; ++s) store_step<XT, L, U>((XT *)a.h + row * g.xs, s, t, g.C, h[s]);
    }
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int s = 0; s < U; ++s) take<XT, NORM>(h[s], gm[s], sum, top);
    uint32_t most = bits_of(top);
    reduce_row<L>(sum, most, red, 0);
    const float rstd = NORM ? rms_factor(sum, g) : 1.0f;
    const Coder code(most);
    // gamma is read again, from the nearest cache, where holding it would cost
    // a wave's place on the unit
    if constexpr (NORM && U > 4) {
        asm volatile("" ::: "memory");
        load_gamma<L, U>(gm, a.gamma, t, g.C);
    }
    if constexpr (NORM)
        if (a.y)
#pragma unroll
            for (int s = 0; s < U; ++s)
                store_step<YT, L, U>((YT *)a.y + row * g.ys, s, t, g.C, normed<XT, YT>(h[s], gm[s], rstd));
    if (!NORM || a.codes)
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const int c = (s * L + t) * kV;
            if (s < full_steps<L, U>() || c < g.stride) store_codes(a.codes + row * g.stride + c, coded<XT, NORM>(h[s], gm[s], code));
        }
    if (t == 0) give_row<NORM>(a, row, rstd, code);
}

// Rows that no block holds, and those of fewer columns than a vector: read twice,
// the second time as the stream if that was written.
template <typename XT, typename YT, bool NORM>
__global__ __launch_bounds__(1024) void k_long_row(RowsGeo g, RmsPtrs a, int blocks) {
    constexpr int L = 1024;
    __shared__ float red[2 * L / 64];
    int b;
    if (!block_number(blocks, b)) return;
    const int64_t row = b;
    const auto fetch = [&](int c, bool again, Vec<XT, kV> &h, Vec<float, kV> &gm) {
        const bool sum = NORM && a.residual && !(again && a.h);
        h = load_any<XT>((const XT *)(NORM && again && a.h ? a.h : a.x) + row * g.xs, c, g.C);
        if (sum) h = add_rounded(h, load_any<XT>((const XT *)a.residual + row * g.xs, c, g.C));
        if constexpr (NORM) {
            if (a.gamma) {
                gm = load_any<float>(a.gamma, c, g.C);
            } else {
#pragma unroll
                for (int k = 0; k < kV; ++k) gm.v[k] = 1.0f;
            }
        }
    };
    float sum = 0.0f, top = 0.0f;
    for (int c = threadIdx.x * kV; c < g.stride; c += L * kV) {
        Vec<XT, kV> h;
        Vec<float, kV> gm;
        fetch(c, false, h, gm);
        if (NORM && a.h && c < g.C) store_cols<XT>((XT *)a.h + row * g.xs, c, g.C, h);
        float part = 0.0f;
        take<XT, NORM>(h, gm, part, top);
        sum += part;
    }
    uint32_t most = bits_of(top);
    reduce_row<L>(sum, most, red, 0);
    const float rstd = NORM ? rms_factor(sum, g) : 1.0f;
    const Coder code(most);
    for (int c = threadIdx.x * kV; c < g.stride; c += L * kV) {
        Vec<XT, kV> h;
        Vec<float, kV> gm;
        fetch(c, true, h, gm);
        if constexpr (NORM)
            if (a.y && c < g.C) store_cols<YT>((YT *)a.y + row * g.ys, c, g.C, normed<XT, YT>(h, gm, rstd));
        if (!NORM || a.codes) store_codes(a.codes + row * g.stride + c, coded<XT, NORM>(h, gm, code));
    }
    if (threadIdx.x == 0) give_row<NORM>(a, row, rstd, code);
}

template <typename XT, typename YT, bool NORM>
void run_rows(const RowsGeo &g, const RmsPtrs &p, hipStream_t st) {
    const int64_t blocks = ((int64_t)g.rows + g.s.per - 1) / g.s.per;
    const auto go = [&](auto kernel, int threads) {
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(threads), 0, st, g, p, (int)blocks);
    };
    if (g.s.lanes == 64) {
        switch (g.s.unroll) {
            case 1: return go(k_row<XT, YT, 64, 1, NORM>, 256);
            case 2: return go(k_row<XT, YT, 64, 2, NORM>, 256);
            case 3: return go(k_row<XT, YT, 64, 3, NORM>, 256);
            case 4: return go(k_row<XT, YT, 64, 4, NORM>, 256);
            case 5: return go(k_row<XT, YT, 64, 5, NORM>, 256);
            case 6: return go(k_row<XT, YT, 64, 6, NORM>, 256);
            default: return go(k_row<XT, YT, 64, 8, NORM>, 256);
        }
    }
    if (g.s.lanes == 256) {
        switch (g.s.unroll) {
            case 3: return go(k_row<XT, YT, 256, 3, NORM>, 256);
            case 4: return go(k_row<XT, YT, 256, 4, NORM>, 256);
            case 5: return go(k_row<XT, YT, 256, 5, NORM>, 256);
            default: return go(k_row<XT, YT, 256, 8, NORM>, 256);
        }
    }
    if (g.s.lanes == 1024) return go(k_row<XT, YT, 1024, 4, NORM>, 1024);
    go(k_long_row<XT, YT, NORM>, 1024);
}

}  // namespace
}  // namespace wq8
