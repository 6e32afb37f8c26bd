// The tiled product of 8-bit codes on matrix cores.
//
// C[m][n] = sum_p 256^-p sum_k A_p(m, k) B(n, k), A in 1, 2 or 4 planes of 8-bit
// digits, both operands with k contiguous in whole lines of 128 bytes, zeros
// behind the last one. A block computes a BM x BN tile in k steps of 128, which
// go from memory to LDS past the registers into one of some buffers while another
// is multiplied: the layout, the swizzle and the loads are those of the bf16
// product, whose k steps have the same bytes. Small tiles, whose blocks are few
// and wait for memory, have three or four buffers, all but one on their way.
// The matrix cores bound it: 8192^3 of random codes in a chain of such calls runs at
// 2400 TOPS (458 us), a library's on the same card at 2270 (485), and
// 16384 x 2560 x 10240 in 411 us (2090 TOPS) before its epilogue.
//
// Two planes are multiplied together, each with sums of its own: what a k step
// has of B serves both, a fragment of it twice the matrix instructions. Of four
// planes the lower two come first; their sum, rounded to the third plane's unit,
// is carried into the second plane's, but for its last byte, which is kept and
// put back at the end. So a block's sums of 2 planes are exact, of 4 to 2^-17 of the
// highest plane's unit. Where k is split the parts of more than one plane are
// rounded to f32 and joined in f32; those of one plane are whole numbers.
#pragma once

#include "wq8_gemm_device.h"
#include "wq8_token_internal.h"

namespace wq8 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Q8Args {
    const int8_t *A, *B;
    int64_t lda, ldb;
    int M, N;
    int steps;         // lines of k
    int tiles_m, tiles_n;
    int ksteps;        // per split
    int splits;
    int64_t plane;     // bytes between planes of A
    void *partial;     // [splits][M][N] where k is split, int32 (one plane) or f32, else NULL
};

// Rows of LDS of a k step, and its buffers: what leaves room for two blocks on a
// compute unit, two at least.
constexpr int q8_rows(int bm, int bn, int planes) { return (planes > 1 ? 2 : 1) * bm + bn; }
constexpr int q8_depth(int rows) { return rows <= 128 ? 4 : rows <= 192 || rows == 384 ? 3 : 2; }
template <int BM, int BN, int PLANES, typename K>
size_t q8_lds(K kernel) {
    constexpr int rows = q8_rows(BM, BN, PLANES);
    constexpr size_t bytes = (size_t)q8_depth(rows) * rows * 128;
    static_assert(bytes <= 163840, "a compute unit's LDS");
    if (bytes > 65536)
        (void)hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return bytes;
}

// Waits until all but the last n of this wave's loads have landed.
template <int n>
__device__ __forceinline__ void wait_all_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

// EPI, an epilogue: column(n) and item(m, n) read what belongs to 8 columns and to
// 8 columns of a row; with(f) calls f once with the activation; store<ACT>(m, n, 8
// sums, span, column, item) ends it: four neighbouring lanes (16 apart) have 32
// columns of a row, and the lanes of the last columns see to what stands behind
// them, `span` being the distance to the columns that no lane has. Each WHOLE:
// all rows and columns of the tile exist (asked for only
// where plain()), or for any m and n.
template <int BM, int BN, int WM, int WN, int PLANES, typename EPI>
__device__ __forceinline__ void q8_block(const Q8Args &a, const EPI &epi, int b, int nb) {
    constexpr int BK = 128, THREADS = WM * WN * 64;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static_assert(TN % 2 == 0, "column tiles come in pairs");
    extern __shared__ __align__(128) char smem[];
    int8_t *const lds = (int8_t *)smem;
    constexpr int NP = PLANES > 1 ? 2 : 1, ROWS = q8_rows(BM, BN, PLANES), STAGE = ROWS * BK, AS = BM * BK, BS = NP * AS;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tiles = a.tiles_m * a.tiles_n;
    b = xcd_block(b, nb);
    const int split = b / tiles, t = b - split * tiles;
    const int band = t / (8 * a.tiles_n), in = t - band * 8 * a.tiles_n;
    const int height = min(8, a.tiles_m - band * 8);
    const int m0 = (band * 8 + in % height) * BM, n0 = (in / height) * BN;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    using SA = Stager<int8_t, true, false, BM, THREADS, false>;
    SA sa = {a.A, a.lda, m0, a.M, 0, 0, 0, {}};
    Stager<int8_t, true, true, BN, THREADS, false> sb = {a.B, a.ldb, n0, a.N, 0, 0, 0, {}};
    sa.prepare();
    sb.prepare();
    const int k0 = split * a.ksteps, k1 = min(k0 + a.ksteps, a.steps), n = k1 - k0;

    i32x4 acc[NP][TM][TN] = {};
    uint32_t rest[PLANES == 4 ? TM : 1][TN];  // the kept bytes of four sums
    const auto multiply = [&](const int8_t *buf) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 fa[NP][TM], fb[TN];
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int row = wm + i * 16 + row_of<false>(lane & 15, 0);
                    fa[p][i] = *(const i32x4 *)(buf + p * AS + lds_unit<int8_t, true, false, BM>(row, kk * 4 + (lane >> 4)));
                }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = wn + (j / 2) * 32 + row_of<true>(lane & 15, j % 2);
                fb[j] = *(const i32x4 *)(buf + BS + lds_unit<int8_t, true, true, BN>(row, kk * 4 + (lane >> 4)));
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[p][i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[p][i], acc[p][i][j], 0, 0, 0);
        }
    };

    // Steps of both passes over the planes, counted through.
    constexpr int D = q8_depth(ROWS), LOADS = NP * SA::COUNT + decltype(sb)::COUNT, PASSES = PLANES / NP;
    const int8_t *plane = a.A + (PLANES - NP) * a.plane;
    int sent = 0, sent_k = 0, to = 0, from = 0, left = n * PASSES;
    const int total = left;
    const auto send = [&] {
        int8_t *const buf = lds + to * STAGE;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            sa.src = plane + p * a.plane;
            sa.direct(buf + p * AS, k0 + sent_k);
        }
        sb.direct(buf + BS, k0 + sent_k);
        to = to + 1 < D ? to + 1 : 0;
        ++sent;
        if (++sent_k == n) {
            sent_k = 0;
            plane -= NP * a.plane;
        }
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        if (d < total) send();
    const auto pass = [&] {
        for (int k = 0; k < n; ++k, --left) {
            if (D == 2 || left < D - 1) wait_all_but<0>();
            else wait_all_but<LOADS *(D - 2)>();
            __syncthreads();
            if (sent < total) send();
            multiply(lds + from * STAGE);
            from = from + 1 < D ? from + 1 : 0;
        }
    };
    pass();
    if constexpr (PLANES == 4) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const i32x4 low = acc[0][i][j] + ((acc[1][i][j] + 128) >> 8);
                rest[i][j] = (low[0] & 255) | (low[1] & 255) << 8 | (low[2] & 255) << 16 | (uint32_t)low[3] << 24;
                acc[0][i][j] = i32x4{};
                acc[1][i][j] = low >> 8;
            }
        pass();
    }

    // the 8 adjacent columns that a lane has in a pair of tiles, in units of the
    // lowest byte that is left
    const auto sums = [&](int i, int j) {
        Vec<float, 8> r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto value = [&](int jj) {
                const float v = (float)acc[0][i][jj][e];
                if constexpr (PLANES == 1) return v;
                const float w = fmaf(v, 256.0f, (float)acc[NP - 1][i][jj][e]);
                if constexpr (PLANES == 2) return w;
                return fmaf(w, 256.0f, (float)(rest[PLANES == 4 ? i : 0][jj] >> (8 * e) & 255));
            };
            r.v[e] = value(j);
            r.v[4 + e] = value(j + 1);
        }
        return r;
    };
    const int mr = m0 + wm + (lane & 15), nc = n0 + wn + (lane >> 4) * 8;
    if (a.partial) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; j += 2) {
                const int m = mr + i * 16, c = nc + j * 16;
                if (m >= a.M || c >= a.N) continue;
                const int64_t at = ((int64_t)split * a.M + m) * a.N + c;
                if constexpr (PLANES > 1) {
                    store_vec_n<float, 8>((float *)a.partial + at, sums(i, j), a.N - c);
                } else {
                    Vec<int, 8> r;
#pragma unroll
                    for (int e = 0; e < 4; ++e) r.v[e] = acc[0][i][j][e], r.v[4 + e] = acc[0][i][j + 1][e];
                    store_vec_n<int, 8>((int *)a.partial + at, r, a.N - c);
                }
            }
        return;
    }
    // what the epilogue reads is on its way a row of tiles ahead
    const auto finish = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        typename EPI::Column col[TN / 2];
        typename EPI::Item next[TN / 2];
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
            col[j] = epi.template column<WHOLE>(nc + j * 32);
            next[j] = epi.template item<WHOLE>(mr, nc + j * 32);
        }
        epi.with([&](auto act) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                typename EPI::Item item[TN / 2];
#pragma unroll
                for (int j = 0; j < TN / 2; ++j) {
                    item[j] = next[j];
                    if (i + 1 < TM) next[j] = epi.template item<WHOLE>(mr + (i + 1) * 16, nc + j * 32);
                }
                // the loads stay in front of the stores: behind them they would wait for these
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < TN / 2; ++j)
                    epi.template store<decltype(act)::value, WHOLE>(mr + i * 16, nc + j * 32, sums(i, 2 * j), a.tiles_n * BN,
                                                                    col[j], item[j]);
            }
        });
    };
    if (m0 + BM <= a.M && n0 + BN <= a.N && epi.plain()) finish(std::true_type{});
    else finish(std::false_type{});
}

template <int BM, int BN, int WM, int WN, int PLANES, typename EPI>
__global__ __launch_bounds__(WM *WN * 64) void k_q8(Q8Args a, EPI epi) {
    int b;
    const int nb = a.tiles_m * a.tiles_n * a.splits;
    if (block_number(nb, b)) q8_block<BM, BN, WM, WN, PLANES>(a, epi, b, nb);
}

// The sum over the splits of 8 columns from n on of row m, those past the end any
// number. Loads stand under no condition, so that some are on their way together:
// they start earlier at a row's end, and the sums are moved to their places.
template <typename T, typename S>
__device__ __forceinline__ void sum_splits(const Q8Args &a, int m, int n, S (&s)[8]) {
    const int64_t size = (int64_t)a.M * a.N;
    const T *const row = (const T *)a.partial + (int64_t)min(m, a.M - 1) * a.N;
    S t[8] = {};
    if (a.N < 8) {
        for (int k = 0; k < a.splits; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += row[k * size + min(n + e, a.N - 1)];
        return;
    }
    const int at = min(n, a.N - 8), shift = n - at;
#pragma unroll 4
    for (int k = 0; k < a.splits; ++k) {
        const Vec<T, 8> v = load_vec<T, 8>(row + k * size + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] += v.v[e];
    }
#pragma unroll
    for (int step = 4; step >= 1; step >>= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const S far = e + step < 8 ? t[e + step < 8 ? e + step : e] : S(0);
            t[e] = (shift & step) ? far : t[e];
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = t[e];
}

// Joins split products in the order of k and runs the epilogue: 32 columns of 16
// rows a wave, 8 columns of a row a lane, as in the product. Whole numbers are
// summed as such.
template <int PLANES, typename EPI>
__device__ __forceinline__ void q8_join_block(const Q8Args &a, const EPI &epi, int b) {
    const int lane = threadIdx.x & 63, ncol = (a.N + 127) / 128;
    const int row = b / ncol, col = b - row * ncol;
    const int m = row * 16 + (lane & 15), n = col * 128 + (threadIdx.x >> 6) * 32 + (lane >> 4) * 8;
    Vec<float, 8> s = {};
    if constexpr (PLANES > 1) {
        sum_splits<float>(a, m, n, s.v);
    } else {
        int64_t t[8] = {};
        sum_splits<int>(a, m, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] = (float)t[e];
    }
    const auto column = epi.template column<false>(n);
    const auto item = epi.template item<false>(m, n);
    epi.with([&](auto act) { epi.template store<decltype(act)::value, false>(m, n, s, ncol * 128, column, item); });
}
inline int64_t q8_join_blocks(const Q8Args &a) {
    return a.splits > 1 ? (int64_t)((a.M + 15) / 16) * ((a.N + 127) / 128) : 0;
}

template <int PLANES, typename EPI>
__global__ __launch_bounds__(256) void k_q8_join(Q8Args a, EPI epi, int nb) {
    int b;
    if (block_number(nb, b)) q8_join_block<PLANES>(a, epi, b);
}

// A product's tiles of BM x BN and its split; returns its blocks.
template <int BM, int BN>
int64_t q8_tiles(Q8Args &a, const Q8Shape &s, void *partial) {
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    a.ksteps = s.ksteps;
    a.splits = s.splits;
    a.partial = s.splits > 1 ? partial : nullptr;
    return (int64_t)a.tiles_m * a.tiles_n * s.splits;
}

// Calls run<BM, BN, WM, WN>() for the tile, in the order of kQ8Tiles, or of
// kQ8PairTiles for more than one plane.
template <typename R>
void pick_q8_tile(int tile, const R &run) {
    switch (tile) {
        case 0: return run.template operator()<256, 256, 2, 4>();
        case 1: return run.template operator()<128, 128, 2, 2>();
        case 2: return run.template operator()<128, 64, 2, 2>();
        default: return run.template operator()<64, 64, 2, 2>();
    }
}
template <typename R>
void pick_q8_pair_tile(int tile, const R &run) {
    switch (tile) {
        case 0: return run.template operator()<256, 128, 4, 2>();
        case 1: return run.template operator()<128, 128, 4, 2>();
        case 2: return run.template operator()<128, 64, 2, 2>();
        default: return run.template operator()<64, 64, 2, 2>();
    }
}

}  // namespace
}  // namespace wq8
