// The tiled product on matrix cores that the linear operator's passes share.
//
// C[m][n] = sum_k A(m, k) B(n, k). A block computes a BM x BN tile, k in steps
// of 128 bytes (64 bf16 or 32 fp32 values). Each operand's step lies in LDS as
// global memory has it: with k contiguous as rows of 128 bytes, with the
// row index contiguous as one row per k. A wave's fragment is 16 bytes per
// lane: lane l holds row l % 16 and the (l / 16)-th 16-byte run of 64 bytes of
// k, which is the bf16 16x16x32 matrix instruction's operand and, element by
// element, that of four fp32 16x16x4 instructions (any order of k serves, as
// long as both operands share it). Where the row index is contiguous, bf16
// fragments come through the transposing LDS read, fp32 ones as single words.
//
// 16-byte units are swizzled in LDS so that a fragment's lanes meet different
// banks: unit u of row r of a k-contiguous tile lies at u ^ (r % 8); in the
// other form units move in pairs (bf16, 32 bytes) or fours (fp32, 64 bytes),
// the extent that 16 lanes read of one k, by the low bits of k that differ
// between the rows of one read.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wq8_device.h"
#include "wq8_ops_device.h"

namespace wq8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct GemmArgs {
    const void *A, *B;
    int64_t lda, ldb;
    int M, N, K;
    int tiles_m, tiles_n;
    int ksteps;        // per split
    float *partial;    // [splits][M][N] where k is split, else NULL
};

// LDS position (in elements) of element (r, k) of an operand tile of R rows
// whose 16-byte unit starts at (r, k).
template <typename T, bool KC, int R>
__device__ __forceinline__ int lds_unit(int row, int unit) {
    constexpr int U = 16 / sizeof(T);
    if constexpr (KC) {  // row: m, unit: along k
        return row * (8 * U) + ((unit ^ (row & 7)) * U);
    } else {             // row: k, unit: along m
        constexpr int UR = R / U;  // units per row
        const int sw = sizeof(T) == 2 ? (((row & 3) | ((row >> 1) & 4)) << 1) & (UR - 1) : (((row >> 2) & 3) << 2) & (UR - 1);
        return row * R + ((unit ^ sw) * U);
    }
}

// Stages one k step of an operand: R rows from r0, k from k0, what lies
// outside rows x kend as zeros.
template <typename T, bool KC, int R, int THREADS>
__device__ __forceinline__ void stage(T *lds, const T *src, int64_t ld, int r0, int rows, int k0, int kend) {
    constexpr int U = 16 / sizeof(T), UNITS = R * 8;
#pragma unroll
    for (int i = 0; i < UNITS / THREADS; ++i) {
        const int q = i * THREADS + threadIdx.x;
        int row, unit, n;
        const T *p;
        if constexpr (KC) {
            row = q / 8;
            unit = q % 8;
            const int k = k0 + unit * U;
            n = r0 + row < rows ? min(kend - k, U) : 0;
            p = src + (int64_t)(r0 + row) * ld + k;
        } else {
            constexpr int UR = R / U;
            row = q / UR;
            unit = q % UR;
            const int m = r0 + unit * U;
            n = k0 + row < kend ? min(rows - m, U) : 0;
            p = src + (int64_t)(k0 + row) * ld + m;
        }
        const Vec<T, U> v = load_vec_n<T, U>(p, n);
        *(Vec<T, U> *)(lds + lds_unit<T, KC, R>(row, unit)) = v;
    }
}

template <typename T>
struct Frag;
template <>
struct Frag<bf16_t> {
    bf16x8 v;
};
template <>
struct Frag<float> {
    f32x4 v;
};

// The fragment of rows r0..r0+15 and the kk-th 64 bytes of k.
template <typename T, bool KC, int R>
__device__ __forceinline__ Frag<T> read_frag(const T *lds, int r0, int kk, int lane) {
    Frag<T> f;
    if constexpr (KC) {
        f.v = *(const decltype(f.v) *)(lds + lds_unit<T, true, R>(r0 + (lane & 15), kk * 4 + (lane >> 4)));
    } else if constexpr (sizeof(T) == 2) {
        // one read gives a lane 4 consecutive k of its row: its group of 16
        // lanes fetches 4 rows of k, 4 lanes and 32 bytes each
        typedef __attribute__((address_space(3))) s16x4 lds4;
        s16x4 h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = kk * 32 + (lane >> 4) * 8 + j * 4 + ((lane & 15) >> 2), m = r0 + (lane & 3) * 4;
            const T *p = lds + lds_unit<T, false, R>(k, m / 8) + m % 8;
            h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
        }
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x8 b = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
        f.v = __builtin_bit_cast(bf16x8, b);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = kk * 16 + (lane >> 4) * 4 + j, m = r0 + (lane & 15);
            f.v[j] = lds[lds_unit<T, false, R>(k, m / 4) + m % 4];
        }
    }
    return f;
}

// acc[i] of lane l: row n = 4 (l / 16) + i of the first operand, row m = l % 16
// of the second.
__device__ __forceinline__ void mma(f32x4 &acc, const Frag<bf16_t> &n, const Frag<bf16_t> &m) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n.v, m.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, const Frag<float> &n, const Frag<float> &m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(n.v[j], m.v[j], acc, 0, 0, 0);
}

// EPI: epilogue(m, n, 4 sums of columns n.., how many of them exist).
template <typename T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, typename EPI>
__global__ __launch_bounds__(WM *WN * 64) void k_gemm(GemmArgs a, EPI epi) {
    constexpr int BK = 128 / sizeof(T), THREADS = WM * WN * 64;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles per wave
    __shared__ __align__(16) T As[BM * BK], Bs[BN * BK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tiles = a.tiles_m * a.tiles_n;
    const int b = xcd_block(blockIdx.x, gridDim.x);
    const int split = b / tiles, t = b % tiles;
    const int m0 = (t / a.tiles_n) * BM, n0 = (t % a.tiles_n) * BN;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    f32x4 acc[TM][TN] = {};
    const int ks = split * a.ksteps, ke = min(ks + a.ksteps, (a.K + BK - 1) / BK);
    for (int s = ks; s < ke; ++s) {
        stage<T, AKC, BM, THREADS>(As, (const T *)a.A, a.lda, m0, a.M, s * BK, a.K);
        stage<T, BKC, BN, THREADS>(Bs, (const T *)a.B, a.ldb, n0, a.N, s * BK, a.K);
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            Frag<T> fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[i] = read_frag<T, AKC, BM>(As, wm + i * 16, kk, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[j] = read_frag<T, BKC, BN>(Bs, wn + j * 16, kk, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) mma(acc[i][j], fb[j], fa[i]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + wm + i * 16 + (lane & 15);
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = n0 + wn + j * 16 + (lane >> 4) * 4;
            if (n >= a.N) continue;
            if (a.partial) {
                Vec<float, 4> r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.v[e] = acc[i][j][e];
                store_vec_n<float, 4>(a.partial + ((int64_t)split * a.M + m) * a.N + n, r, a.N - n);
            } else {
                epi(m, n, acc[i][j], a.N - n);
            }
        }
    }
}

// Joins split products, in the order of k, and runs the epilogue: a thread per
// 4 columns of a row.
template <typename EPI>
__global__ __launch_bounds__(256) void k_gemm_join(GemmArgs a, int splits, EPI epi) {
    const int nq = (a.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.M * nq) return;
    const int m = (int)(i / nq), n = (int)(i % nq) * 4;
    f32x4 s = {};
    for (int k = 0; k < splits; ++k) {
        const Vec<float, 4> v = load_vec_n<float, 4>(a.partial + ((int64_t)k * a.M + m) * a.N + n, a.N - n);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v.v[e];
    }
    epi(m, n, s, a.N - n);
}

template <typename T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, typename EPI>
void run_tile(const GemmShape &s, GemmArgs a, const EPI &epi, float *partial, hipStream_t st) {
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    a.ksteps = s.ksteps;
    a.partial = s.splits > 1 ? partial : nullptr;
    const unsigned blocks = (unsigned)((int64_t)a.tiles_m * a.tiles_n * s.splits);
    hipLaunchKernelGGL((k_gemm<T, AKC, BKC, BM, BN, WM, WN, EPI>), dim3(blocks), dim3(WM * WN * 64), 0, st, a, epi);
    if (s.splits > 1) {
        const int64_t work = (int64_t)a.M * ((a.N + 3) / 4);
        hipLaunchKernelGGL((k_gemm_join<EPI>), dim3((unsigned)((work + 255) / 256)), dim3(256), 0, st, a, s.splits, epi);
    }
}

template <typename T, bool AKC, bool BKC, typename EPI>
void run_gemm(const GemmShape &s, const GemmArgs &a, const EPI &epi, float *partial, hipStream_t st) {
    if (a.M == 0 || a.N == 0) return;
    run_tile<T, AKC, BKC, 128, 128, 2, 2>(s, a, epi, partial, st);
}

}  // namespace
}  // namespace wq8
