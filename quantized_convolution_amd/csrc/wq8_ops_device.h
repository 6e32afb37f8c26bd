// Device helpers of the group norm and the matrix product: activations with
// their derivatives, bf16 conversion, vectors of any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "wq8_device.h"
#include "wq8_ops_internal.h"

namespace wq8 {

typedef uint16_t bf16_t;  // bf16 bits
typedef __bf16 hw_bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Nearest even; a NaN stays a NaN.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
    return __builtin_bit_cast(bf16_t, (__bf16)v);
}

// Grids: a launch takes fewer than 2^32 threads in a dimension (more are cut
// off without an error), so blocks of up to 1024 threads stand in rows of 2^21.
constexpr unsigned kGridRow = 1u << 21;
inline dim3 grid_of(int64_t blocks) {
    return blocks <= kGridRow ? dim3((unsigned)blocks) : dim3(kGridRow, (unsigned)((blocks + kGridRow - 1) / kGridRow));
}
// This block's number; false for those that fill the last row up.
__device__ __forceinline__ bool block_number(int blocks, int &b) {
    b = (int)(blockIdx.y * kGridRow + blockIdx.x);
    return (unsigned)b < (unsigned)blocks;
}

// V adjacent elements. Loads and stores copy bytes, so the address need only
// be aligned to the element: the target takes unaligned 4- to 16-byte global
// accesses in one instruction.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
    Vec<T, V> r;
    __builtin_memcpy(&r, p, sizeof r);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &r) {
    __builtin_memcpy(p, &r, sizeof r);
}
// The first n of V elements, the rest zero (n <= 0: all zero, nothing read). A
// part of a vector takes one access per set bit of n.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec_n(const T *p, int n) {
    Vec<T, V> r = {};
    if (n >= V) return load_vec<T, V>(p);
    if constexpr (V > 1) {
        constexpr int H = V / 2;
        if (n >= H) {
            const Vec<T, H> lo = load_vec<T, H>(p), hi = load_vec_n<T, H>(p + H, n - H);
#pragma unroll
            for (int i = 0; i < H; ++i) r.v[i] = lo.v[i], r.v[H + i] = hi.v[i];
        } else if (n > 0) {
            const Vec<T, H> lo = load_vec_n<T, H>(p, n);
#pragma unroll
            for (int i = 0; i < H; ++i) r.v[i] = lo.v[i];
        }
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec_n(T *p, const Vec<T, V> &r, int n) {
    if (n >= V) {
        store_vec<T, V>(p, r);
    } else if constexpr (V > 1) {
        constexpr int H = V / 2;
        Vec<T, H> lo, hi;
#pragma unroll
        for (int i = 0; i < H; ++i) lo.v[i] = r.v[i], hi.v[i] = r.v[H + i];
        if (n >= H) {
            store_vec<T, H>(p, lo);
            store_vec_n<T, H>(p + H, hi, n - H);
        } else if (n > 0) {
            store_vec_n<T, H>(p, lo, n);
        }
    }
}

// ------------------------------------------------------------- activations
// EXACT: to some roundings of fp32, for results in fp32. Else, for bf16 ones,
// whose own rounding is 2^-9, in fewer instructions: relative errors of |z|
// 2^-24 in the exponentials, 1.5e-7 absolute in gelu's distribution function.
// For bf16 the exact forms cost 815 -> 865 us at a product of 16384 x 2560 x 10240
// with gelu and 18.7 -> 21.3 us at a norm's backward of 8 x 640 x 32 x 32 with silu;
// the short ones would save fp32 0.7 of 7.8 us at a norm of 8 x 1280 x 16 x 16 and
// 1.0 of 28.9 at a backward of 2 x 320 x 64 x 64.
template <typename X, typename Y>
constexpr bool exact_acts() { return sizeof(X) == 4 || sizeof(Y) == 4; }

// exp(x + lo), on the hardware's 2^x (1 ulp). EXACT, for x <= 0: 2^n 2^f, |f| <=
// 1/2, with n and f of the unrounded x log2(e), denormal results among them.
template <bool EXACT>
__device__ __forceinline__ float exp_of(float x, float lo = 0.0f) {
    constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = 1.925963033e-8f;
    if constexpr (!EXACT) return __builtin_amdgcn_exp2f(x * kLog2e);
    x = fmaxf(x, -150.0f);  // 0 from there on
    const float n = __builtin_rintf(x * kLog2e), f = fmaf(lo, kLog2e, fmaf(x, kLog2eRest, fmaf(x, kLog2e, -n)));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }  // 1 ulp, no denormals

// 1 / (1 + exp(-z)) and what it leaves of 1. EXACT: both small ends without
// cancellation; not the function's value for a NaN: the activations multiply
// it by z.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z, float *rest) {
    if constexpr (EXACT) {
        const float e = exp_of<true>(-fabsf(z)), r = fast_rcp(1.0f + e), er = e * r;
        *rest = z >= 0.0f ? er : r;
        return z >= 0.0f ? r : er;
    } else {
        const float s = fast_rcp(1.0f + exp_of<false>(-z));
        *rest = 1.0f - s;
        return s;
    }
}

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2), from
// Phi(-|z|) = e r P(r) with r a reciprocal linear in |z|.
// EXACT: P of degree 8 in (x - 2) / (x + 2), x = |z| / sqrt 2, of 0.5 (x + 2)
// erfc(x) exp(x^2), fitted for the least relative error over |z| <= 13.5
// (4.3e-8; the mapping of the half line is Shepherd and Laframboise's, Math.
// Comp. 36, 1981): within 7 2^-24 of Phi(-|z|), relative, evaluated in fp32.
// Else: Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26.
template <bool EXACT>
__device__ __forceinline__ float normal_cdf(float z, float *e_out) {
    float e, q;
    if constexpr (EXACT) {
        const float a = fminf(fabsf(z), 30.0f), h = a * a;  // 30: e is 0 from there on
        e = exp_of<true>(-0.5f * h, -0.5f * fmaf(a, a, -h));
        const float r = fast_rcp(a + 2.82842712475f), t = fmaf(-5.65685424949f, r, 1.0f);
        float s = fmaf(-0.000325433502f, t, -0.000532054051f);
        s = fmaf(s, t, 0.0021066654f);
        s = fmaf(s, t, 0.00455091987f);
        s = fmaf(s, t, -0.0151914684f);
        s = fmaf(s, t, -0.0257634148f);
        s = fmaf(s, t, 0.197614923f);
        s = fmaf(s, t, -0.4858962f);
        s = fmaf(s, t, 0.722368062f);
        q = r * s * e;
    } else {
        e = exp_of<false>(-0.5f * z * z);
        const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.0f));
        float s = fmaf(1.061405429f, t, -1.453152027f);
        s = fmaf(s, t, 1.421413741f);
        s = fmaf(s, t, -0.284496736f);
        s = fmaf(s, t, 0.254829592f);
        q = 0.5f * s * t * e;
    }
    *e_out = e;
    return z >= 0.0f ? 1.0f - q : (z < 0.0f ? q : z);  // NaN stays NaN
}

constexpr float kGeluTanh2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// z * gate, where a gate of 0 comes from z running to -infinity: the limit of
// every activation there is 0, and -infinity itself gives NaN (-inf * 0).
template <int ACT, bool EXACT>
__device__ __forceinline__ float act_fwd(float z) {
    if constexpr (ACT == WQ8_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    float rest;
    if constexpr (ACT == WQ8_ACT_SILU) return z * sigmoid<EXACT>(z, &rest);
    if constexpr (ACT == WQ8_ACT_GELU) return z * normal_cdf<EXACT>(z, &rest);
    if constexpr (ACT == WQ8_ACT_GELU_TANH)  // (1 + tanh u) / 2 = sigmoid(2 u)
        return z * sigmoid<EXACT>(kGeluTanh2 * fmaf(kGeluCubic * z * z, z, z), &rest);
    return z;
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == WQ8_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    float rest;
    if constexpr (ACT == WQ8_ACT_SILU) {
        const float s = sigmoid<EXACT>(z, &rest);
        return s * fmaf(z, rest, 1.0f);
    }
    if constexpr (ACT == WQ8_ACT_GELU) {
        const float c = normal_cdf<EXACT>(z, &rest);
        return fmaf(z * 0.3989422804014327f, rest, c);
    }
    if constexpr (ACT == WQ8_ACT_GELU_TANH) {
        const float s = sigmoid<EXACT>(kGeluTanh2 * fmaf(kGeluCubic * z * z, z, z), &rest);
        // s rest is 0 long before z^2 overflows: 0 times infinity would be a NaN
        const float b = __builtin_amdgcn_fmed3f(z, -1e9f, 1e9f);
        return fmaf(z * s * rest, kGeluTanh2 * fmaf(3.0f * kGeluCubic * b, b, 1.0f), s);
    }
    return 1.0f;
}

// f(act) with the run-time activation as a constant, so that the choice is
// one uniform branch around a loop and not one per element.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case WQ8_ACT_RELU: f(std::integral_constant<int, WQ8_ACT_RELU>{}); break;
        case WQ8_ACT_SILU: f(std::integral_constant<int, WQ8_ACT_SILU>{}); break;
        case WQ8_ACT_GELU: f(std::integral_constant<int, WQ8_ACT_GELU>{}); break;
        case WQ8_ACT_GELU_TANH: f(std::integral_constant<int, WQ8_ACT_GELU_TANH>{}); break;
        default: f(std::integral_constant<int, WQ8_ACT_NONE>{}); break;
    }
}

// v of the lane that the DPP control names.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the 64 lanes, in all of them.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<kDppXor1>(v);
    v += dpp<kDppXor2>(v);
    v += dpp<kDppXor7>(v);  // the other half of 8: quads already agree
    v += dpp<kDppXor8>(v);
    const auto r16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r16[0]) + __uint_as_float(r16[1]);
    const auto r32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r32[0]) + __uint_as_float(r32[1]);
}

}  // namespace wq8
