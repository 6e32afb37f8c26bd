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
// exp(x) on the hardware's 2^x: the argument's rounding gives a relative
// error of |x| 2^-24, below 1e-6 where the result matters to an activation.
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }  // 1 ulp

__device__ __forceinline__ float sigmoid(float z) { return fast_rcp(1.0f + fast_exp(-z)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2).
// Phi(-|z|) = poly(t) e / 2 with t = 1 / (1 + p |z| / sqrt 2): Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26 (|error of erf| <=
// 1.5e-7, fp32's own at these sizes), a third of the library erf's
// instructions.
__device__ __forceinline__ float normal_cdf(float z, float *e_out) {
    const float e = fast_exp(-0.5f * z * z);
    const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.0f));
    float s = fmaf(1.061405429f, t, -1.453152027f);
    s = fmaf(s, t, 1.421413741f);
    s = fmaf(s, t, -0.284496736f);
    s = fmaf(s, t, 0.254829592f);
    const float q = 0.5f * s * t * e;
    *e_out = e;
    return z >= 0.0f ? 1.0f - q : (z < 0.0f ? q : z);  // NaN stays NaN
}

constexpr float kGeluTanh2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// z * gate, where a gate of 0 comes from z running to -infinity: the limit of
// every activation there is 0, and -infinity itself gives NaN (-inf * 0).
template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
    if constexpr (ACT == WQ8_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == WQ8_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == WQ8_ACT_GELU) {
        float e;
        return z * normal_cdf(z, &e);
    }
    if constexpr (ACT == WQ8_ACT_GELU_TANH)  // (1 + tanh u) / 2 = sigmoid(2 u)
        return z * sigmoid(kGeluTanh2 * fmaf(kGeluCubic * z * z, z, z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == WQ8_ACT_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == WQ8_ACT_SILU) {
        const float s = sigmoid(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == WQ8_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, &e);
        return fmaf(z * 0.3989422804014327f, e, c);
    }
    if constexpr (ACT == WQ8_ACT_GELU_TANH) {
        const float s = sigmoid(kGeluTanh2 * fmaf(kGeluCubic * z * z, z, z));
        return fmaf(z * s * (1.0f - s), kGeluTanh2 * fmaf(3.0f * kGeluCubic * z, z, 1.0f), s);
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
