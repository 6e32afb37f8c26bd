// Device helpers of the kernels that hold rows in registers: columns by
// vectors of 8, reductions over a row's threads, codes.
#pragma once

#include "wq8_ops_device.h"
#include "wq8_token_internal.h"

namespace wq8 {
namespace {

constexpr int kV = 8;  // columns of a thread in one step: 16 bytes of bf16, a quarter of a group's 32 codes

// Columns [c, c + 8) of a row of C >= 8, zeros from C on. The load stands under
// no condition of its own: it starts earlier at a row's end, and what belongs to
// other columns is shifted out.
template <typename T>
__device__ __forceinline__ Vec<T, kV> load_cols(const T *row, int c, int C) {
    const int at = min(c, C - kV), shift = c - at;
    Vec<T, kV> r = load_vec<T, kV>(row + at);
    if (C % kV == 0) {
        if (shift) r = Vec<T, kV>{};
        return r;
    }
    if (shift) {  // one lane of a row's, and those behind it
#pragma unroll
        for (int step = 4; step >= 1; step >>= 1)
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                const T v = k + step < kV ? r.v[k + step < kV ? k + step : k] : T(0);
                r.v[k] = shift >= kV ? T(0) : (shift & step) ? v : r.v[k];
            }
    }
    return r;
}

// The same for any C.
template <typename T>
__device__ __forceinline__ Vec<T, kV> load_any(const T *row, int c, int C) {
    if (C >= kV) return load_cols<T>(row, c, C);
    Vec<T, kV> r;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
        const T v = row[min(c + k, C - 1)];
        r.v[k] = c + k < C ? v : T(0);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store_cols(T *row, int c, int C, const Vec<T, kV> &v) {
    store_vec_n<T, kV>(row + c, v, C - c);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    const auto step = [&](int other) { v = max(v, (uint32_t)other); };
    step(__builtin_amdgcn_update_dpp(0, (int)v, kDppXor1, 0xf, 0xf, true));
    step(__builtin_amdgcn_update_dpp(0, (int)v, kDppXor2, 0xf, 0xf, true));
    step(__builtin_amdgcn_update_dpp(0, (int)v, kDppXor7, 0xf, 0xf, true));
    step(__builtin_amdgcn_update_dpp(0, (int)v, kDppXor8, 0xf, 0xf, true));
    const auto r16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r16[0], r16[1]);
    const auto r32 = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(r32[0], r32[1]);
}

__device__ __forceinline__ int wave_add(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, kDppXor1, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kDppXor2, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kDppXor7, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kDppXor8, 0xf, 0xf, true);
    const auto r16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = (int)r16[0] + (int)r16[1];
    const auto r32 = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (int)r32[0] + (int)r32[1];
}

// The larger magnitude of m >= 0 and v; a NaN stays.
__device__ __forceinline__ float larger(float m, float v) { return __builtin_elementwise_maximum(m, __builtin_fabsf(v)); }
__device__ __forceinline__ float largest(const float (&v)[kV]) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < kV; ++k) m = larger(m, v[k]);
    return m;
}
// Its bits: as whole numbers they order as magnitudes do, infinities above all
// finite ones and NaN above those.
__device__ __forceinline__ uint32_t bits_of(float m) { return __float_as_uint(m) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kInv127 = 1.0f / 127.0f;

// How values of largest magnitude `a` (its bits) become codes: code = rint((x up) f).
struct Coder {
    float up, f, scale;
    bool bad;

    __device__ __forceinline__ explicit Coder(uint32_t bits) {
        const float a = __uint_as_float(bits);
        bad = false;
        up = 1.0f;
        if (__builtin_expect(!__any(!(a >= 0x1p-100f && a < 0x1p100f)), 1)) {
            // Both quotients as division rounds them (all significands checked; the
            // exponent does not matter here), in 9 operations for some 24: an
            // approximation, and what it leaves times the reciprocal (Markstein, IBM
            // J. Res. Dev. 34, 1990).
            float y = fast_rcp(a);
            y = fmaf(fmaf(-a, y, 1.0f), y, y);
            const float q = 127.0f * y, s = a * kInv127;
            f = fmaf(fmaf(-a, q, 127.0f), y, q);
            scale = fmaf(fmaf(-127.0f, s, a), kInv127, s);
            return;
        }
        bad = bits >= kInfBits;
        up = a < 0x1p-100f ? 0x1p64f : 1.0f;  // 127 / a overflows below 2^-121
        f = bits == 0 ? 0.0f : 127.0f / (a * up);
        scale = bad ? __uint_as_float(0x7fc00000u) : a / 127.0f;
    }
    // |(x up) f| <= 127 (1 + 2^-24)^2 < 127.5, so its nearest whole number is a code
    __device__ __forceinline__ uint64_t pack(const float (&x)[kV]) const {
        float t[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) t[k] = x[k];
        if (__builtin_expect(__any(up != 1.0f), 0))  // times one is left out
#pragma unroll
            for (int k = 0; k < kV; ++k) t[k] *= up;
#pragma unroll
        for (int k = 0; k < kV; ++k) t[k] = t[k] * f + kRoundMagic;
        const uint32_t lo = pack4(t[0], t[1], t[2], t[3]), hi = pack4(t[4], t[5], t[6], t[7]);
        return bad ? 0 : (uint64_t)hi << 32 | lo;
    }
};

__device__ __forceinline__ void store_codes(int8_t *p, uint64_t v) { *(uint64_t *)p = v; }

// Sum and largest over the threads of a row: a wave, or a block of L threads.
// `turn` alternates between two halves of `red` where a block calls it again and
// again, so that one barrier each is enough.
template <int L>
__device__ __forceinline__ void reduce_row(float &sum, uint32_t &most, float *red, int turn) {
    sum = wave_sum(sum);
    most = wave_max(most);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        float *const r = red + (turn & 1) * 2 * W;
        if ((threadIdx.x & 63) == 0) {
            r[threadIdx.x >> 6] = sum;
            r[W + (threadIdx.x >> 6)] = __uint_as_float(most);
        }
        __syncthreads();
        sum = 0.0f;
        most = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            sum += r[w];
            most = max(most, __float_as_uint(r[W + w]));
        }
    }
}

// Steps of a row held by L threads in U steps that lie in it whole, by the widths
// that the plan gives that shape: the others alone look for the row's end.
template <int L, int U>
constexpr int full_steps() {
    return L == 1024 && U == 4 ? 2 : U == 8 ? (L == 64 ? 6 : 5) : U - 1;
}

template <typename T, int L, int U>
__device__ __forceinline__ void load_row(Vec<T, kV> (&v)[U], const T *row, int t, int C) {
#pragma unroll
    for (int s = 0; s < U; ++s)
        v[s] = s < full_steps<L, U>() ? load_vec<T, kV>(row + (s * L + t) * kV) : load_cols<T>(row, (s * L + t) * kV, C);
}

template <int L, int U>
__device__ __forceinline__ void load_gamma(Vec<float, kV> (&v)[U], const float *gamma, int t, int C) {
    if (gamma) return load_row<float, L, U>(v, gamma, t, C);
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
        for (int k = 0; k < kV; ++k) v[s].v[k] = 1.0f;
}

// Columns c of step s, which lies in the row whole or may pass its end.
template <typename T, int L, int U>
__device__ __forceinline__ void store_step(T *row, int s, int t, int C, const Vec<T, kV> &v) {
    const int c = (s * L + t) * kV;
    if (s < full_steps<L, U>()) store_vec<T, kV>(row + c, v);
    else if (c < C) store_cols<T>(row, c, C, v);
}

}  // namespace
}  // namespace wq8
