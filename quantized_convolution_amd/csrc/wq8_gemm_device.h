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
// banks (see swizzle()).
//
// What bounds it: bf16, the matrix cores' clock under load and, for tiles below
// 256 x 256, LDS reads (a wave of 64 x 64 reads as long as it multiplies).
// 8192^3 runs at 1337 TFLOP/s in 256 x 256 tiles, 1150 in 128 x 128; a library
// product of that size reaches 1392. fp32: the matrix instruction, 146 of 154
// TFLOP/s at 8192 x 4096 x 4096. Small products: filling 256 compute units, which
// is what the choice of tile and split weighs, and the first loads' latency.
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
    int splits;
    int more;          // 1: A is the sum of two matrices, `plane` elements apart;
    int64_t plane;     // each k step is taken once for each
    float *partial;    // [splits][M][N] where k is split, else NULL
};

// Where a tile keeps its 16-byte units. `unit` runs along the contiguous
// dimension of row `row` (k contiguous: row = m or n; otherwise row = k).
// FIRST: the operand whose rows become the sums' columns (B, see kRowOf).
template <typename T, bool KC, bool FIRST, int R>
__device__ __forceinline__ int swizzle(int row, int unit) {
    constexpr int UR = KC ? 8 : R / (16 / (int)sizeof(T));  // units per row
    if constexpr (KC) {
        // 16 lanes read one unit of 16 rows (128 bytes apart): spread them over
        // the 16 units of 256 bytes, two rows' worth. B's rows are 8a + b.
        const int s = FIRST ? ((row >> 1) & 1) | ((row >> 2) & 6) : (row >> 1) & 7;
        return unit ^ s;
    } else if constexpr (sizeof(T) == 2) {
        return unit ^ ((((row & 3) | ((row >> 1) & 4)) << 1) & (UR - 1));
    } else {
        return unit ^ ((((row >> 2) & 3) << 2) & (UR - 1));
    }
}

template <typename T, bool KC, bool FIRST, int R>
__device__ __forceinline__ int lds_unit(int row, int unit) {
    constexpr int U = 16 / sizeof(T);
    return row * (KC ? 8 * U : R) + swizzle<T, KC, FIRST, R>(row, unit) * U;
}

// Stages k steps of an operand of R tile rows. Units that lie in LDS one after
// another are one thread each, so a wave's 64 units can be one load from
// memory to LDS; the swizzle is in the address that a thread reads.
// TWO: the operand, or the other one, may be the sum of two matrices.
template <typename T, bool KC, bool FIRST, int R, int THREADS, bool TWO>
struct Stager {
    static constexpr int U = 16 / sizeof(T), UR = KC ? 8 : R / U, COUNT = R * 8 / THREADS, BK = 128 / sizeof(T);
    static_assert(R * 8 % THREADS == 0, "whole waves");

    const T *src;
    int64_t ld;
    int r0, rows, K;
    int more;
    int64_t plane;
    uint32_t off[COUNT];

    // Steps count the matrices within k steps, so that what both meet in the
    // other operand is still in the cache the second time.
    __device__ __forceinline__ const T *matrix(int &step) const {
        if constexpr (!TWO) return src;
        const T *m = src + (step & more) * plane;
        step >>= more;
        return m;
    }

    __device__ __forceinline__ static void place(int i, int &row, int &unit) {
        const int q = i * THREADS + threadIdx.x;
        row = q / UR;
        unit = swizzle<T, KC, FIRST, R>(row, q % UR);
    }

    // Byte offsets of the direct loads from the tile's first element of a step.
    // Rows past the end repeat the last one: their sums are not stored. Needs
    // 16-byte aligned rows, and whole units along the rows' index.
    __device__ __forceinline__ void prepare() {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            int row, unit;
            place(i, row, unit);
            if constexpr (KC) off[i] = (uint32_t)(min(row, rows - 1 - r0) * (uint32_t)ld + unit * U) * (uint32_t)sizeof(T);
            else off[i] = (uint32_t)(row * (uint32_t)ld + min(unit * U, rows - U - r0)) * (uint32_t)sizeof(T);
        }
    }

    // One whole step from memory to LDS, past the registers.
    __device__ __forceinline__ void direct(T *lds, int step) const {
        const T *const mat = matrix(step);
        const T *base = KC ? mat + (int64_t)r0 * ld + (int64_t)step * BK : mat + (int64_t)step * BK * ld + r0;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, -1, kBufferFlags);
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) T *)lds + (threadIdx.x >> 6) * 1024;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            const uint32_t m0 = __builtin_amdgcn_readfirstlane(at + i * THREADS * 16);
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"(m0), "v"(off[i]), "s"(r)
                         : "memory");
        }
    }

    // A step through registers, at any alignment, in loads without conditions (a
    // load under one is waited for before the next is sent). Rows past the end
    // hold anything: their sums are not stored.
    //
    // Whether a step needs no care: all of its k exist, and where the rows' index
    // is the contiguous one a unit that passes the rows' end reads on into the
    // next k's row, so that must exist as well.
    __device__ __forceinline__ bool whole(int step) const {
        if constexpr (TWO) step >>= more;
        return KC ? (step + 1) * BK <= K : (step + 1) * BK < K && rows >= U;
    }
    __device__ __forceinline__ void load(Vec<T, U> (&v)[COUNT], int step) const {
        const T *const mat = matrix(step);
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            int row, unit;
            place(i, row, unit);
            if constexpr (KC) v[i] = load_vec<T, U>(mat + (int64_t)min(r0 + row, rows - 1) * ld + step * BK + unit * U);
            else v[i] = load_vec<T, U>(mat + (int64_t)(step * BK + row) * ld + min(r0 + unit * U, rows - 1));
        }
    }
    // The last step: zeros for k past the end. A unit that passes the end of
    // its row is read from U before that end and moved down.
    __device__ __forceinline__ void load_last(Vec<T, U> (&v)[COUNT], int step) const {
        const int end = KC ? K : rows;  // of the contiguous index
        const T *const mat = matrix(step);
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            int row, unit;
            place(i, row, unit);
            const int at = (KC ? step * BK : r0) + unit * U, line = KC ? r0 + row : step * BK + row;
            const int lines = KC ? rows : K;
            const T *p = mat + (int64_t)min(line, lines - 1) * ld;
            const int n = KC || line < lines ? end - at : 0;  // values that count
            if (end >= U) {
                const int from = min(at, end - U), shift = at - from;
                const Vec<T, U> r = load_vec<T, U>(p + from);
#pragma unroll
                for (int e = 0; e < U; ++e) {
                    T x = T(0);
#pragma unroll
                    for (int q = e; q < U; ++q) x = q - e == shift ? r.v[q] : x;
                    v[i].v[e] = e < n ? x : T(0);
                }
            } else {
                v[i] = load_vec_n<T, U>(p + at, n);
            }
        }
    }
    __device__ __forceinline__ void store(T *lds, const Vec<T, U> (&v)[COUNT]) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) *(Vec<T, U> *)(lds + (i * THREADS + threadIdx.x) * U) = v[i];
    }
};

// Waits until this wave's direct loads have landed in LDS.
__device__ __forceinline__ void wait_direct() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

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

// Row of a fragment's lane r = l % 16. A: consecutive rows. B: tile pairs share
// 32 columns, the even one taking the first 4 of every 8 and the odd one the
// last, so that a lane's sums of both are 8 adjacent columns.
template <bool FIRST>
__device__ __forceinline__ int row_of(int r, int odd) {
    return FIRST ? (r >> 2) * 8 + (r & 3) + odd * 4 : r;
}

// The fragment of the tile rows from r0 and the kk-th 64 bytes of k.
template <typename T, bool KC, bool FIRST, int R>
__device__ __forceinline__ Frag<T> read_frag(const T *lds, int r0, int odd, int kk, int lane) {
    Frag<T> f;
    if constexpr (KC) {
        const int row = r0 + row_of<FIRST>(lane & 15, odd);
        f.v = *(const decltype(f.v) *)(lds + lds_unit<T, true, FIRST, R>(row, kk * 4 + (lane >> 4)));
    } else if constexpr (sizeof(T) == 2) {
        // one read gives a lane 4 consecutive k of its row: its group of 16
        // lanes fetches 4 rows of k, 4 lanes and 4 runs of 8 bytes each
        typedef __attribute__((address_space(3))) s16x4 lds4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        s16x4 h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = kk * 32 + (lane >> 4) * 8 + j * 4 + ((lane & 15) >> 2), m = r0 + row_of<FIRST>((lane & 3) * 4, odd);
            const T *p = lds + lds_unit<T, false, FIRST, R>(k, m / 8) + m % 8;
            h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
        }
        const s16x8 b = __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
        f.v = __builtin_bit_cast(bf16x8, b);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = kk * 16 + (lane >> 4) * 4 + j, m = r0 + row_of<FIRST>(lane & 15, odd);
            f.v[j] = lds[lds_unit<T, false, FIRST, R>(k, m / 4) + m % 4];
        }
    }
    return f;
}

// acc[i] of lane l: row 4 (l / 16) + i of the first operand (B, the columns n),
// row l % 16 of the second (A, the rows m). fp32: the e-th of 4 instructions.
constexpr int mma_parts(size_t size) { return size == 2 ? 1 : 4; }
__device__ __forceinline__ void mma(f32x4 &acc, const Frag<bf16_t> &n, const Frag<bf16_t> &m, int) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n.v, m.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, const Frag<float> &n, const Frag<float> &m, int e) {
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(n.v[e], m.v[e], acc, 0, 0, 0);
}

// EPI, an epilogue: column(n) and item(m, n) read, for any m and n, what belongs
// to 8 columns and to 8 columns of a row; with(f) calls f once with the
// activation; store<ACT>(m, n, 8 sums, how many exist, column, item) ends it.
// DIRECT: whole k steps go from memory to LDS without registers; a last partial
// one, and every one of operands that are not aligned for that, goes through
// registers. Two buffers: while one is multiplied the other is filled.
// The 8 adjacent columns that a lane has in a pair of tiles.
__device__ __forceinline__ Vec<float, 8> sums(const f32x4 &even, const f32x4 &odd) {
    Vec<float, 8> r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = even[e], r.v[4 + e] = odd[e];
    return r;
}

// The b-th of a product's nb blocks.
template <typename T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, bool DIRECT, bool TWO, typename EPI>
__device__ __forceinline__ void gemm_block(const GemmArgs &a, const EPI &epi, int b, int nb) {
    constexpr int BK = 128 / sizeof(T), THREADS = WM * WN * 64;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles per wave
    static_assert(TN % 2 == 0, "column tiles come in pairs");
    extern __shared__ __align__(128) char smem[];
    T *const lds = (T *)smem;
    constexpr int STAGE = (BM + BN) * BK, BS = BM * BK;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tiles = a.tiles_m * a.tiles_n;
    b = xcd_block(b, nb);
    const int split = b / tiles, t = b - split * tiles;
    // tiles in bands of 8 rows of tiles: blocks that run together share panels
    const int band = t / (8 * a.tiles_n), in = t - band * 8 * a.tiles_n;
    const int height = min(8, a.tiles_m - band * 8);
    const int m0 = (band * 8 + in % height) * BM, n0 = (in / height) * BN;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    Stager<T, AKC, false, BM, THREADS, TWO> sa = {(const T *)a.A, a.lda, m0, a.M, a.K, a.more, a.plane, {}};
    Stager<T, BKC, true, BN, THREADS, TWO> sb = {(const T *)a.B, a.ldb, n0, a.N, a.K, a.more, 0, {}};
    if constexpr (DIRECT) {
        sa.prepare();
        sb.prepare();
    }
    const int k0 = split * a.ksteps, k1 = min(k0 + a.ksteps, (a.K + BK - 1) / BK);
    const int more = TWO ? a.more : 0, ks = k0 << more, ke = k1 << more;
    const int kd = DIRECT ? min(k1, a.K / BK) << more : ks;  // steps [ks, kd) are whole and direct

    f32x4 acc[TM][TN] = {};
    const auto multiply = [&](const T *buf) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            Frag<T> fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[i] = read_frag<T, AKC, false, BM>(buf, wm + i * 16, 0, kk, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j] = read_frag<T, BKC, true, BN>(buf + BS, wn + (j / 2) * 32, j % 2, kk, lane);
#pragma unroll
            for (int e = 0; e < mma_parts(sizeof(T)); ++e)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) mma(acc[i][j], fb[j], fa[i], e);
        }
    };

    int s = ks;
    if (DIRECT && s < kd) {
        sa.direct(lds, s);
        sb.direct(lds + BS, s);
        for (; s < kd; ++s) {
            T *const cur = lds + ((s - ks) & 1) * STAGE, *const nxt = lds + ((s - ks + 1) & 1) * STAGE;
            wait_direct();
            __syncthreads();
            if (s + 1 < kd) {
                sa.direct(nxt, s + 1);
                sb.direct(nxt + BS, s + 1);
            }
            multiply(cur);
        }
    }
    if (s < ke) {
        Vec<T, 16 / sizeof(T)> va[decltype(sa)::COUNT], vb[decltype(sb)::COUNT];
        const auto fetch = [&](int step) {
            if (!DIRECT && sa.whole(step) && sb.whole(step)) {
                sa.load(va, step);
                sb.load(vb, step);
            } else {
                sa.load_last(va, step);
                sb.load_last(vb, step);
            }
        };
        fetch(s);
        for (; s < ke; ++s) {
            T *const cur = lds + ((s - ks) & 1) * STAGE;
            sa.store(cur, va);
            sb.store(cur + BS, vb);
            __syncthreads();
            if (s + 1 < ke) fetch(s + 1);
            multiply(cur);
        }
    }

    if (a.partial) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; j += 2) {
                const int m = m0 + wm + i * 16 + (lane & 15), n = n0 + wn + j * 16 + (lane >> 4) * 8;
                if (m < a.M && n < a.N)
                    store_vec_n<float, 8>(a.partial + ((int64_t)split * a.M + m) * a.N + n, sums(acc[i][j], acc[i][j + 1]),
                                          a.N - n);
            }
        return;
    }
    // what the epilogue reads is on its way a row of tiles ahead
    const int mr = m0 + wm + (lane & 15), nc = n0 + wn + (lane >> 4) * 8;
    typename EPI::Column col[TN / 2];
    typename EPI::Item next[TN / 2];
#pragma unroll
    for (int j = 0; j < TN / 2; ++j) {
        col[j] = epi.column(nc + j * 32);
        next[j] = epi.item(mr, nc + j * 32);
    }
    epi.with([&](auto act) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            typename EPI::Item item[TN / 2];
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                item[j] = next[j];
                if (i + 1 < TM) next[j] = epi.item(mr + (i + 1) * 16, nc + j * 32);
            }
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                const int m = mr + i * 16, n = nc + j * 32;
                if (m < a.M && n < a.N)
                    epi.template store<decltype(act)::value>(m, n, sums(acc[i][2 * j], acc[i][2 * j + 1]), a.N - n, col[j],
                                                             item[j]);
            }
        }
    });
}

template <typename T, bool AKC, bool BKC, int BM, int BN, int WM, int WN, bool DIRECT, typename EPI>
__global__ __launch_bounds__(WM *WN * 64) void k_gemm(GemmArgs a, EPI epi) {
    int b;
    const int nb = a.tiles_m * a.tiles_n * a.splits;
    if (block_number(nb, b)) gemm_block<T, AKC, BKC, BM, BN, WM, WN, DIRECT, false>(a, epi, b, nb);
}

// Joins split products, in the order of k, and runs the epilogue. A thread takes
// 8 columns of a row and a wave 32 columns of 16 rows, as in the product: whole
// 128-byte runs of the sums, and 16 adjacent pixels of an NCHW residual.
// 2048 x 1280 fp32 in two parts with an NCHW residual: 9.5 us for 42 MB.
template <typename EPI>
__device__ __forceinline__ void join_block(const GemmArgs &a, const EPI &epi, int b) {
    const int lane = threadIdx.x & 63, ncol = (a.N + 127) / 128;
    const int row = b / ncol, col = b - row * ncol;
    const int m = row * 16 + (lane & 15), n = col * 128 + (threadIdx.x >> 6) * 32 + (lane >> 4) * 8;
    if (m >= a.M || n >= a.N) return;
    Vec<float, 8> s = {};
    for (int k = 0; k < a.splits; ++k) {
        const Vec<float, 8> v = load_vec_n<float, 8>(a.partial + ((int64_t)k * a.M + m) * a.N + n, a.N - n);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] += v.v[e];
    }
    const auto column = epi.column(n);
    const auto item = epi.item(m, n);
    epi.with([&](auto act) { epi.template store<decltype(act)::value>(m, n, s, a.N - n, column, item); });
}
inline int64_t join_blocks(const GemmArgs &a) {
    return a.splits > 1 ? (int64_t)((a.M + 15) / 16) * ((a.N + 127) / 128) : 0;
}

template <typename EPI>
__global__ __launch_bounds__(256) void k_gemm_join(GemmArgs a, EPI epi, int nb) {
    int b;
    if (block_number(nb, b)) join_block(a, epi, b);
}

// A product's tiles of BM x BN and its split; returns its blocks.
template <int BM, int BN>
int64_t set_tiles(GemmArgs &a, const GemmShape &s, float *partial) {
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    a.ksteps = s.ksteps;
    a.splits = s.splits;
    a.partial = s.splits > 1 ? partial : nullptr;
    return (int64_t)a.tiles_m * a.tiles_n * s.splits;
}

// Bytes of LDS of a tile, allowed for `kernel` where they pass the default.
template <int BM, int BN, typename K>
size_t tile_lds(K kernel) {
    constexpr size_t bytes = 2 * (BM + BN) * 128;
    if (bytes > 65536)
        (void)hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return bytes;
}

// Calls run<BM, BN, WM, WN, DIRECT>() for tile s.tile, in the order of
// kGemmTiles. Not DIRECT, the largest tile has no registers for a step; the
// plan does not choose it then, nor 128 x 128 for SMALL.
template <bool SMALL, typename R>
void pick_tile(const GemmShape &s, const R &run) {
    const auto go = [&](auto direct) {
        constexpr bool D = decltype(direct)::value;
        switch (s.tile) {
            case 0:
                if constexpr (D) run.template operator()<256, 256, 2, 4, D>();
                return;
            case 1:
                if constexpr (!SMALL) run.template operator()<128, 128, 2, 2, D>();
                return;
            case 2: return run.template operator()<128, 64, 2, 2, D>();
            case 3: return run.template operator()<64, 64, 2, 2, D>();
            default: return run.template operator()<16, 128, 1, 2, D>();
        }
    };
    if (s.direct) go(std::true_type{});
    else go(std::false_type{});
}

}  // namespace
}  // namespace wq8
