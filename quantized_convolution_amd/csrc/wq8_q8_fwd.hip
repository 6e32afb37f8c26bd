// Matrix product of 8-bit codes with scales for each token and channel:
//   z = (xq wq^T) sx sw + bias;  y = act(z) + residual
// The sums are whole numbers on the int8 matrix cores; scales, bias, activation,
// residual and what is kept of z (as it is, or in codes of 32 columns, which
// four lanes of a wave have) are in the epilogue.
//
// Up to four rows (single tokens) have a kernel of their own.
#include "wq8_q8_gemm.h"
#include "wq8_rows.h"

namespace wq8 {
namespace {

static __device__ const float kNothing[8] = {};

// gelu for bf16 results, z Phi(z) = max(z, 0) - |z| Phi(-|z|), with Phi(-|z|) as
// normal_cdf<false>() has it, its half taken into the coefficients: 12 operations
// and two transcendental ones for 20. The bound on |z| keeps infinity times 0 out.
__device__ __forceinline__ float gelu_of(float z) {
    const float a = fminf(fabsf(z), 1e18f), e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);  // exp(-z^2 / 2)
    const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752f, a, 1.0f));
    float s = fmaf(0.5307027145f, t, -0.7265760135f);
    s = fmaf(s, t, 0.7107068705f);
    s = fmaf(s, t, -0.142248368f);
    s = fmaf(s, t, 0.127414796f);
    return fmaf(-a, s * t * e, fmaxf(z, 0.0f));
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == WQ8_ACT_GELU && !EXACT) return gelu_of(z);
    return act_fwd<ACT, EXACT>(z);
}

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

    // Whether whole tiles have nothing that is read across their rows. (With both
    // kinds of residual in one body the compiler reads either by single values.)
    __device__ __forceinline__ bool plain() const { return !(planar && residual); }

    // Rows and columns past the end read the last ones' values, and what is not
    // given reads zeros, so that loads stand under no condition but one for all.
    template <bool WHOLE>
    __device__ __forceinline__ Column column(int n) const {
        Column c = {};
        if constexpr (WHOLE) {
            if (bias) c.bias = load_vec<float, 8>(bias + n);
            c.sw = load_vec<float, 8>(sw + n);
        } else if (N % 8 == 0) {
            c.bias = load_vec<float, 8>(bias ? bias + min(n, N - 8) : kNothing);
            c.sw = load_vec<float, 8>(sw + min(n, N - 8));
        } else {
            c.bias = load_vec_n<float, 8>(bias + n, bias ? N - n : 0);
            c.sw = load_vec_n<float, 8>(sw + n, N - n);
        }
        return c;
    }

    template <bool WHOLE>
    __device__ __forceinline__ Item item(int m, int n) const {
        Item r = {};
        const int row = min(m, M - 1);
        r.sx = sx[row];
        if constexpr (WHOLE) {
            if (residual) r.residual = load_vec<YT, 8>(residual + row * rs + n);
        } else if (planar && residual) {
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

    template <bool WHOLE>
    __device__ __forceinline__ void put(YT *p, int n, const Vec<float, 8> &v) const {
        Vec<YT, 8> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = from_f32<YT>(v.v[e]);
        if constexpr (WHOLE) store_vec<YT, 8>(p, r);
        else store_vec_n<YT, 8>(p, r, N - n);
    }

    template <int ACT, bool WHOLE>
    __device__ __forceinline__ void store(int m, int n, Vec<float, 8> v, int span, const Column &col, const Item &item) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = v.v[e] * item.sx * col.sw.v[e];
        if (bias)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += col.bias.v[e];
        if (zq) {  // all lanes: a group's four meet
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = v.v[e];
            if (!WHOLE && N % 32 != 0)  // else a group's columns exist all or none
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = n + e < N ? t[e] : 0.0f;
            uint32_t most = bits_of(largest(t));
            const auto r16 = __builtin_amdgcn_permlane16_swap(most, most, false, false);
            most = max(r16[0], r16[1]);
            const auto r32 = __builtin_amdgcn_permlane32_swap(most, most, false, false);
            most = max(r32[0], r32[1]);
            const Coder code(most);
            if (WHOLE || m < M) {
                int8_t *const to = zq + (int64_t)m * Np;
                if (WHOLE || n < Np) store_codes(to + n, WHOLE || n < N ? code.pack(t) : 0);
                for (int c = n + span; c < Np; c += span) store_codes(to + c, 0);
                if (n % 32 == 0 && (WHOLE || n < N)) sz[(int64_t)m * ((N + 31) / 32) + n / 32] = code.scale;
            }
        }
        if (!WHOLE && (m >= M || n >= N)) return;
        if (z) put<WHOLE>(z + (int64_t)m * N + n, n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = act_of<ACT, exact_acts<YT, YT>()>(v.v[e]);
        if (residual)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.v[e] += to_f32(item.residual.v[e]);
        put<WHOLE>(y + (int64_t)m * ys + n, n, v);
    }
};

// Up to 4 rows: each weight is used so few times that it needs no matrix core,
// and reads best along its row. A wave takes 4096 bytes of a weight row at a
// time, 16 a lane, four products an instruction, OUT columns in turn, two of them
// with their loads in flight; the rows' codes stay in registers meanwhile. Sums
// over the lanes are whole numbers, in any order the same.
constexpr int kDotWaves = 4;

template <int ROWS, int OUT, typename EPI>
__global__ __launch_bounds__(kDotWaves * 64) void k_q8_dot(Q8Args a, EPI epi, int blocks) {
    constexpr int CHUNK = 4, COLS = kDotWaves * OUT, PAIR = 2;
    __shared__ int sums[ROWS][COLS];
    int b;
    if (!block_number(blocks, b)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = b * COLS;
    const int bytes = a.steps * 128;
#pragma unroll 1
    for (int o = 0; o < OUT; o += PAIR) {
        const int8_t *w[PAIR];
#pragma unroll
        for (int j = 0; j < PAIR; ++j) w[j] = a.B + (int64_t)min(n0 + wave * OUT + o + j, a.N - 1) * a.ldb;
        int acc[PAIR][ROWS] = {};
        for (int k0 = 0; k0 < bytes; k0 += CHUNK * 1024) {
            i32x4 v[PAIR][CHUNK], x[ROWS][CHUNK];
#pragma unroll
            for (int c = 0; c < CHUNK; ++c) {
                const int k = k0 + c * 1024 + lane * 16, at = min(k, bytes - 16);
#pragma unroll
                for (int j = 0; j < PAIR; ++j) v[j][c] = *(const i32x4 *)(w[j] + at);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) x[r][c] = *(const i32x4 *)(a.A + (int64_t)min(r, a.M - 1) * a.lda + at);
                if (k != at)  // past the end: counted by the lane that has it
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) x[r][c] = i32x4{};
            }
#pragma unroll
            for (int c = 0; c < CHUNK; ++c)
#pragma unroll
                for (int j = 0; j < PAIR; ++j)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][r] = __builtin_amdgcn_sdot4(v[j][c][e], x[r][c][e], acc[j][r], false);
        }
#pragma unroll
        for (int j = 0; j < PAIR; ++j)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int t = wave_add(acc[j][r]);
                if (lane == 0) sums[r][wave * OUT + o + j] = t;
            }
    }
    __syncthreads();
    if (wave > 0) return;
    const int g = lane >> 4, n = n0 + g * 8;
    const int m = g * 8 < COLS && (lane & 15) < ROWS ? (lane & 15) : a.M;
    Vec<float, 8> v = {};
    if (m < a.M)
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = (float)sums[m][g * 8 + e];
    epi.with([&](auto act) {
        epi.template store<decltype(act)::value, false>(m, n, v, blocks * COLS, epi.template column<false>(n),
                                                        epi.template item<false>(m, n));
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
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(WM * WN * 64), (q8_lds<BM, BN, 1>(kernel)), st, a, epi());
        if (a.splits > 1)
            hipLaunchKernelGGL((k_q8_join<1, EpiQ8<YT>>), grid_of(q8_join_blocks(a)), dim3(256), 0, st, a, epi(),
                               (int)q8_join_blocks(a));
    }

    template <int ROWS>
    void few() const {
        const auto go = [&](auto kernel, int cols) {
            const int blocks = (g.N + cols - 1) / cols;
            hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(kDotWaves * 64), 0, st, args(), epi(), blocks);
        };
        // codes of z need their 32 columns in one block; else 8 spread evenly
        // over the compute units
        if (p.zq) go(k_q8_dot<ROWS, 8, EpiQ8<YT>>, 32);
        else go(k_q8_dot<ROWS, 2, EpiQ8<YT>>, 8);
    }

    void run() const {
        if (g.f.tile >= 0) return pick_q8_tile(g.f.tile, *this);
        if (g.M == 1) few<1>();
        else if (g.M == 2) few<2>();
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
