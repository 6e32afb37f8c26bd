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

// The bits of |v|: as whole numbers they order as the magnitudes do, infinities
// above all finite ones and NaN above those.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// How values of largest magnitude `a` (its bits) become codes: code = rint((x up) f).
struct Coder {
    float up, f, scale;
    bool bad;

    __device__ __forceinline__ explicit Coder(uint32_t bits) {
        const float a = __uint_as_float(bits);
        bad = bits >= kInfBits;
        up = a < 0x1p-100f ? 0x1p64f : 1.0f;  // 127 / a overflows below 2^-121
        f = bits == 0 ? 0.0f : 127.0f / (a * up);
        scale = bad ? __uint_as_float(0x7fc00000u) : a / 127.0f;
    }
    // |(x up) f| <= 127 (1 + 2^-24)^2 < 127.5, so its nearest whole number is a code
    __device__ __forceinline__ float raw(float x) const { return x * up * f + kRoundMagic; }
    __device__ __forceinline__ uint64_t pack(const float (&x)[kV]) const {
        const uint32_t lo = pack4(raw(x[0]), raw(x[1]), raw(x[2]), raw(x[3]));
        const uint32_t hi = pack4(raw(x[4]), raw(x[5]), raw(x[6]), raw(x[7]));
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

// f(lanes, unroll) for the shape, both as constants.
template <int L, int U>
struct RowConst {
    static constexpr int lanes = L, unroll = U;
};

}  // namespace
}  // namespace wq8
