// Matrix product of 8-bit codes with scales for each token and channel:
//   z = (xq wq^T) sx sw + bias;  y = act(z) + residual
// The sums are whole numbers on the int8 matrix cores; scales, bias, activation,
// residual and what is kept of z (as it is, or in codes of 32 columns, which
// four lanes of a wave have) are in the epilogue.
//
// A few rows (one token, a short batch) have a kernel of their own: it only has
// to stream the weights, so its waves read their fragments from memory past LDS,
// 16 or 32 columns a block, the waves of a block along k.
#include "wq8_q8_gemm.h"
#include "wq8_rows.h"

namespace wq8 {
namespace {

static __device__ const float kNothing[8] = {};

template <typename YT>
struct EpiQ8 {
    const float *bias, *sx, *sw;
    const YT *residual;
    YT *y, *z;
    int8_t *zq;
    float *sz;
    int64_t ys, rs;
    int M, N, Np, act, planar, pixels;

    struct Column {
        Vec<float, 8> bias, sw;
    };
    struct Item {
        Vec<YT, 8> residual;
        float sx;
    };

    // Rows and columns past the end read the last ones' values, and what is not
    // given reads zeros, so that loads stand under no condition but one for all.
    __device__ __forceinline__ Column column(int n) const {
        Column c;
        if (N % 8 == 0) {
            c.bias = load_vec<float, 8>(bias ? bias + min(n, N - 8) : kNothing);
            c.sw = load_vec<float, 8>(sw + min(n, N - 8));
        } else {
            c.bias = load_vec_n<float, 8>(bias + n, bias ? N - n : 0);
            c.sw = load_vec_n<float, 8>(sw + n, N - n);
        }
        return c;
    }

    __device__ __forceinline__ Item item(int m, int n) const {
        Item r;
        const int row = min(m, M - 1);
        r.sx = sx[row];
        if (planar && residual) {
            const int img = row / pixels, p = row - img * pixels;
            const YT *src = residual + (int64_t)img * N * pixels + p;
#pragma unroll
            for (int e = 0; e < 8; ++e) r.residual.v[e] = src[(int64_t)min(n + e, N - 1) * pixels];
        } else if (N % 8 == 0) {
            r.residual = load_vec<YT, 8>(residual ? residual + row * rs + min(n, N - 8) : (const YT *)kNothing);
        } else {
            r.residual = load_vec_n<YT, 8>(residual + row * rs + n, residual ? N - n : 0);
        }
        return r;
    }

    template <typename F>
    __device__ __forceinline__ void with(F f) const {
        with_act(act, f);
    }

    template <int ACT>
    __device__ __forceinline__ void store(int m, int n, Vec<float, 8> v, int span, const Column &col, const Item &item) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = v.v[e] * item.sx * col.sw.v[e];
        if (bias)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += col.bias.v[e];
        if (zq) {  // all lanes: a group's four meet
            float t[8];
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[e] = n + e < N ? v.v[e] : 0.0f;
                most = max(most, magnitude(t[e]));
            }
            const auto r16 = __builtin_amdgcn_permlane16_swap(most, most, false, false);
            most = max(r16[0], r16[1]);
            const auto r32 = __builtin_amdgcn_permlane32_swap(most, most, false, false);
            most = max(r32[0], r32[1]);
            const Coder code(most);
            if (m < M) {
                int8_t *const to = zq + (int64_t)m * Np;
                if (n < Np) store_codes(to + n, code.pack(t));
                for (int c = n + span; c < Np; c += span) store_codes(to + c, 0);
                if (n % 32 == 0 && n < N) sz[(int64_t)m * ((N + 31) / 32) + n / 32] = code.scale;
            }
        }
        if (m >= M || n >= N) return;
        Vec<YT, 8> r;
        if (z) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
            store_vec_n<YT, 8>(z + (int64_t)m * N + n, r, N - n);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = act_fwd<ACT, exact_acts<YT, YT>()>(v.v[e]);
        if (residual)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += to_f32(item.residual.v[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
        store_vec_n<YT, 8>(y + (int64_t)m * ys + n, r, N - n);
    }
};

// MT tiles of 16 rows, 32 columns a block, W waves along k. A wave's fragment
// is 16 rows of 64 adjacent bytes; two of them make its lines whole, so a wave
// takes steps of 128 bytes, every W-th. Rows and columns past the end repeat the
// last one.
template <int MT, int W, typename EPI>
__global__ __launch_bounds__(W * 64) void k_q8_few(Q8Args a, EPI epi, int blocks) {
    constexpr int DEPTH = MT == 1 ? 4 : 2;  // steps whose loads are in flight together
    __shared__ i32x4 red[W > 1 ? W : 1][MT][2][64];
    int b;
    if (!block_number(blocks, b)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n0 = b * 32;
    const int8_t *pa[MT], *pb[2];
#pragma unroll
    for (int i = 0; i < MT; ++i) pa[i] = a.A + (int64_t)min(i * 16 + (lane & 15), a.M - 1) * a.lda + (lane >> 4) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) pb[j] = a.B + (int64_t)min(n0 + row_of<true>(lane & 15, j), a.N - 1) * a.ldb + (lane >> 4) * 16;
    i32x4 acc[MT][2] = {};
    for (int s = wave; s < a.steps; s += W * DEPTH) {
        i32x4 fa[DEPTH][MT][2], fb[DEPTH][2][2];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int64_t k = (int64_t)min(s + d * W, a.steps - 1) * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < 2; ++j) fb[d][j][h] = *(const i32x4 *)(pb[j] + k + h * 64);
#pragma unroll
                for (int i = 0; i < MT; ++i) fa[d][i][h] = *(const i32x4 *)(pa[i] + k + h * 64);
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (s + d * W < a.steps)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[d][j][h], fa[d][i][h], acc[i][j], 0, 0, 0);
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) red[wave][i][j][lane] = acc[i][j];
        __syncthreads();
    }
    const int n = n0 + (lane >> 4) * 8;
    epi.with([&](auto act) {
        for (int i = wave; i < MT; i += W) {  // a wave joins a tile of rows
            i32x4 t[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (W > 1) {
                    t[j] = red[0][i][j][lane];
#pragma unroll
                    for (int w = 1; w < W; ++w) t[j] += red[w][i][j][lane];
                } else {
                    t[j] = acc[i][j];
                }
            }
            const int m = i * 16 + (lane & 15);
            Vec<float, 8> v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v.v[e] = (float)t[0][e], v.v[4 + e] = (float)t[1][e];
            epi.template store<decltype(act)::value>(m, n, v, blocks * 32, epi.column(n), epi.item(m, n));
        }
    });
}

template <typename YT>
struct RunQ8 {
    const Q8Geo &g;
    const Q8Ptrs &p;
    hipStream_t st;

    EpiQ8<YT> epi() const {
        return {p.bias, p.sx, p.sw, (const YT *)p.residual, (YT *)p.y, (YT *)p.z, p.zq, p.sz, g.ys, g.rs, g.M, g.N, g.Np, g.act,
                g.r_planar, g.pixels};
    }
    Q8Args args() const {
        Q8Args a = {};
        a.A = p.xq;
        a.B = p.wq;
        a.lda = a.ldb = g.Kp;
        a.M = g.M;
        a.N = g.N;
        a.steps = g.Kp / 128;
        return a;
    }

    template <int BM, int BN, int WM, int WN>
    void operator()() const {
        Q8Args a = args();
        const int64_t blocks = q8_tiles<BM, BN>(a, g.f, p.partial);
        const auto kernel = k_q8<BM, BN, WM, WN, 1, EpiQ8<YT>>;
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(WM * WN * 64), (tile_lds<BM, BN>(kernel)), st, a, epi());
        if (a.splits > 1)
            hipLaunchKernelGGL((k_q8_join<1, EpiQ8<YT>>), grid_of(q8_join_blocks(a)), dim3(256), 0, st, a, epi(),
                               (int)q8_join_blocks(a));
    }

    template <int MT>
    void few() const {
        const int blocks = (g.N + 31) / 32;
        const auto go = [&](auto kernel, int w) {
            hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(w * 64), 0, st, args(), epi(), blocks);
        };
        if (g.few_waves == 4) go(k_q8_few<MT, 4, EpiQ8<YT>>, 4);
        else go(k_q8_few<MT, 8, EpiQ8<YT>>, 8);
    }

    void run() const {
        if (g.f.tile >= 0) return pick_q8_tile<false>(g.f.tile, *this);
        if (g.few_rows == 1) few<1>();
        else if (g.few_rows == 2) few<2>();
        else few<4>();
    }
};

}  // namespace

wq8_status launch_q8_forward(const Q8Geo &g, wq8_dtype ydt, const Q8Ptrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (ydt == WQ8_F32) RunQ8<float>{g, p, st}.run();
    else RunQ8<bf16_t>{g, p, st}.run();
    return check_launch("product of codes");
}

}  // namespace wq8
