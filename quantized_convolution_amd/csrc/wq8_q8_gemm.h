// The tiled product of 8-bit codes on matrix cores.
//
// C[m][n] = sum_p 256^-p sum_k A_p(m, k) B(n, k), A in 1, 2 or 4 planes of 8-bit
// digits, both operands with k contiguous in whole lines of 128 bytes, zeros
// behind the last one. A block computes a BM x BN tile in k steps of 128, which
// go from memory to LDS past the registers into one of two buffers while the
// other is multiplied: the layout, the swizzle and the loads are those of the
// bf16 product, whose k steps have the same bytes.
//
// Several planes share the sums' registers. The lowest comes first; after each
// but the highest a sum is shifted down by 8 bits and the next plane is added to
// what is left. The bits that the shifts drop are kept in a byte each and put
// back at the end, so the sums of 2 planes are exact; of 4 planes the lowest 8
// bits, below 2^-16 of the highest plane's unit, are rounded off.
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

// EPI, an epilogue: column(n) and item(m, n) read, for any m and n, what belongs
// to 8 columns and to 8 columns of a row; with(f) calls f once with the
// activation; store<ACT>(m, n, 8 sums, span, column, item) ends it, for any m
// and n: four neighbouring lanes (16 apart) have 32 columns of a row, and the
// lanes of the last columns see to what stands behind them, `span` being the
// distance to the columns that no lane has.
template <int BM, int BN, int WM, int WN, int PLANES, typename EPI>
__device__ __forceinline__ void q8_block(const Q8Args &a, const EPI &epi, int b, int nb) {
    constexpr int BK = 128, THREADS = WM * WN * 64;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static_assert(TN % 2 == 0, "column tiles come in pairs");
    extern __shared__ __align__(128) char smem[];
    int8_t *const lds = (int8_t *)smem;
    constexpr int STAGE = (BM + BN) * BK, BS = BM * BK;
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

    i32x4 acc[TM][TN] = {};
    constexpr int KEPT = PLANES / 2;  // bytes of a sum that shifts have dropped
    uint32_t rest[KEPT ? KEPT : 1][TM][TN];  // the p-th of four sums
    const auto multiply = [&](const int8_t *buf) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = wm + i * 16 + row_of<false>(lane & 15, 0);
                fa[i] = *(const i32x4 *)(buf + lds_unit<int8_t, true, false, BM>(row, kk * 4 + (lane >> 4)));
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int row = wn + (j / 2) * 32 + row_of<true>(lane & 15, j % 2);
                fb[j] = *(const i32x4 *)(buf + BS + lds_unit<int8_t, true, true, BN>(row, kk * 4 + (lane >> 4)));
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    };

    int s = 0;  // steps of all planes, counted through
    sa.src = a.A + (PLANES - 1) * a.plane;
    if (n > 0) {
        sa.direct(lds, k0);
        sb.direct(lds + BS, k0);
    }
    const auto add_plane = [&](bool last) {
        for (int k = 0; k < n; ++k, ++s) {
            int8_t *const cur = lds + (s & 1) * STAGE, *const nxt = lds + ((s + 1) & 1) * STAGE;
            wait_direct();
            __syncthreads();
            if (k + 1 < n) {
                sa.direct(nxt, k0 + k + 1);
                sb.direct(nxt + BS, k0 + k + 1);
            } else if (!last) {
                sa.src -= a.plane;
                sa.direct(nxt, k0);
                sb.direct(nxt + BS, k0);
            }
            multiply(cur);
        }
    };
    if constexpr (PLANES == 4) {
        add_plane(false);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = (acc[i][j] + 128) >> 8;
    }
#pragma unroll
    for (int q = KEPT - 1; q >= 0; --q) {
        add_plane(false);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const i32x4 v = acc[i][j];
                rest[q][i][j] = (v[0] & 255) | (v[1] & 255) << 8 | (v[2] & 255) << 16 | (uint32_t)v[3] << 24;
                acc[i][j] = v >> 8;
            }
    }
    add_plane(true);

    // the 8 adjacent columns that a lane has in a pair of tiles
    const auto sums = [&](int i, int j) {
        Vec<float, 8> r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const auto value = [&](int jj) {  // in units of the lowest byte kept
                const float v = (float)acc[i][jj][e];
                if constexpr (PLANES == 2) return fmaf(v, 256.0f, (float)(rest[0][i][jj] >> (8 * e) & 255));
                if constexpr (PLANES == 4)
                    return fmaf(v, 65536.0f,
                                (float)((rest[0][i][jj] >> (8 * e) & 255) << 8 | (rest[KEPT - 1][i][jj] >> (8 * e) & 255)));
                return v;
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
                    for (int e = 0; e < 4; ++e) r.v[e] = acc[i][j][e], r.v[4 + e] = acc[i][j + 1][e];
                    store_vec_n<int, 8>((int *)a.partial + at, r, a.N - c);
                }
            }
        return;
    }
    // what the epilogue reads is on its way a row of tiles ahead
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
            for (int j = 0; j < TN / 2; ++j)
                epi.template store<decltype(act)::value>(mr + i * 16, nc + j * 32, sums(i, 2 * j), a.tiles_n * BN, col[j],
                                                         item[j]);
        }
    });
}

template <int BM, int BN, int WM, int WN, int PLANES, typename EPI>
__global__ __launch_bounds__(WM *WN * 64) void k_q8(Q8Args a, EPI epi) {
    int b;
    const int nb = a.tiles_m * a.tiles_n * a.splits;
    if (block_number(nb, b)) q8_block<BM, BN, WM, WN, PLANES>(a, epi, b, nb);
}

// Joins split products in the order of k and runs the epilogue: 32 columns of 16
// rows a wave, 8 columns of a row a lane, as in the product. Whole numbers are
// summed as such.
template <int PLANES, typename EPI>
__device__ __forceinline__ void q8_join_block(const Q8Args &a, const EPI &epi, int b) {
    const int lane = threadIdx.x & 63, ncol = (a.N + 127) / 128;
    const int row = b / ncol, col = b - row * ncol;
    const int m = row * 16 + (lane & 15), n = col * 128 + (threadIdx.x >> 6) * 32 + (lane >> 4) * 8;
    const bool in = m < a.M && n < a.N;
    Vec<float, 8> s = {};
    if constexpr (PLANES > 1) {
        for (int k = 0; k < a.splits; ++k) {
            const Vec<float, 8> v =
                load_vec_n<float, 8>((const float *)a.partial + ((int64_t)k * a.M + m) * a.N + n, in ? a.N - n : 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) s.v[e] += v.v[e];
        }
    } else {
        int64_t t[8] = {};
        for (int k = 0; k < a.splits; ++k) {
            const Vec<int, 8> v = load_vec_n<int, 8>((const int *)a.partial + ((int64_t)k * a.M + m) * a.N + n, in ? a.N - n : 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += v.v[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s.v[e] = (float)t[e];
    }
    const auto column = epi.column(n);
    const auto item = epi.item(m, n);
    epi.with([&](auto act) { epi.template store<decltype(act)::value>(m, n, s, ncol * 128, column, item); });
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

// Calls run<BM, BN, WM, WN>() for the tile, in the order of kQ8Tiles.
template <bool MULTI, typename R>
void pick_q8_tile(int tile, const R &run) {
    switch (tile) {
        case 0:
            if constexpr (!MULTI) run.template operator()<256, 256, 2, 4>();
            return;
        case 1: return run.template operator()<128, 128, 2, 2>();
        case 2: return run.template operator()<128, 64, 2, 2>();
        case 3: return run.template operator()<64, 64, 2, 2>();
        default:
            if constexpr (!MULTI) run.template operator()<16, 128, 1, 2>();
    }
}

}  // namespace
}  // namespace wq8
