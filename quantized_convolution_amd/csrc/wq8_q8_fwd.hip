// Matrix product of 8-bit codes with scales for each token and channel:
//   z = (xq wq^T) sx sw + bias;  y = act(z) + residual
// The sums are whole numbers on the int8 matrix cores; scales, bias, activation,
// residual and what is kept of z (as it is, or in codes of 32 columns, which
// four lanes of a wave have) are in the epilogue. With gelu, z in codes and y in bf16
// 16384 x 2560 x 10240 takes 513 to 538 us, without either 410, in fp32 586 and 475:
// the epilogue of the largest tile runs alone on its compute unit.
//
// One or two rows (single tokens) and short batches have kernels of their own.
#include "wq8_q8_gemm.h"
#include "wq8_rows.h"

namespace wq8 {
namespace {

static __device__ const float kNothing[8] = {};

// gelu for bf16 results, z Phi(z) = max(z, 0) - |z| Phi(-|z|), with Phi(-|z|) as
// normal_cdf<false>() has it, its half taken into the coefficients: 12 operations
// and two transcendental ones for 20. The bound keeps infinity times 0 out where z is
// +infinity; -infinity gives a NaN as act_fwd() does.
__device__ __forceinline__ float gelu_of(float z) {
    const float a = fabsf(fminf(z, 1e18f)), e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);  // exp(-z^2 / 2)
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

// One or two rows: each weight is used so few times that it needs no matrix core,
// and reads best along its row. A wave takes 4096 bytes of a weight row at a
// time, 16 a lane, four products an instruction, OUT columns in turn, two of them
// with their loads in flight; the rows' codes stay in registers meanwhile. Sums
// over the lanes are whole numbers, in any order the same. Memory bounds it: one row
// by 10240 x 10240 takes 17.8 to 19.4 us in a chain of such calls (5.4 to 5.9 TB/s),
// 33.7 in a tile.
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

// A short batch: blocks of 16 or 32 rows by 32 columns whose four waves take every
// fourth k step each, so that few steps follow one another. A wave loads its own
// lines of both operands into buffers of its own and waits for no other; the
// sums of the four, whole numbers, meet at the end. 16 rows of 10240 x 10240 take
// 18.8 to 21.6 us, 4.9 to 5.6 TB/s of weights, and 23.8 in a tile whose k steps are
// split over blocks; 64 rows of 1280 x 1280 3.8 us, of which 2.2 are the launch, and 5.7 in
// the smallest tile, whose ten steps follow one another.
constexpr int kThinWaves = 4, kThinCols = 32;
constexpr int thin_depth(int rt) { return rt == 1 ? 3 : 2; }  // two blocks fit a compute unit
constexpr int thin_lds(int rt) { return kThinWaves * thin_depth(rt) * (rt * 16 + kThinCols) * 128; }

template <int RT, typename EPI>
__global__ __launch_bounds__(kThinWaves * 64) void k_q8_thin(Q8Args a, EPI epi, int blocks) {
    constexpr int D = thin_depth(RT), AROWS = RT * 16, STAGE = (AROWS + kThinCols) * 128, AL = AROWS / 8, BL = kThinCols / 8;
    extern __shared__ __align__(128) char smem[];
    int b;
    if (!block_number(blocks, b)) return;
    b = xcd_block(b, blocks);  // blocks of the same columns behind one cache
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tm = (a.M + AROWS - 1) / AROWS, col = b / tm, m0 = (b - col * tm) * AROWS, n0 = col * kThinCols;
    int8_t *const lds = (int8_t *)smem + wave * D * STAGE;
    uint32_t off[AL + BL];
#pragma unroll
    for (int i = 0; i < AL + BL; ++i) {  // 8 rows of 128 bytes a load
        const bool first = i < AL;
        const int row = (first ? i : i - AL) * 8 + (lane >> 3);
        const int unit = first ? swizzle<int8_t, true, false, 16>(row, lane & 7) : swizzle<int8_t, true, true, 16>(row, lane & 7);
        off[i] = first ? (uint32_t)min(row, a.M - 1 - m0) * (uint32_t)a.lda + unit * 16
                       : (uint32_t)min(row, a.N - 1 - n0) * (uint32_t)a.ldb + unit * 16;
    }
    const int n = (a.steps - wave + kThinWaves - 1) / kThinWaves;  // of this wave
    const auto send = [&](int i) {
        const int64_t k = (int64_t)(wave + i * kThinWaves) * 128;
        const __amdgpu_buffer_rsrc_t ra =
            __builtin_amdgcn_make_buffer_rsrc((void *)(a.A + (int64_t)m0 * a.lda + k), 0, -1, kBufferFlags);
        const __amdgpu_buffer_rsrc_t rb =
            __builtin_amdgcn_make_buffer_rsrc((void *)(a.B + (int64_t)n0 * a.ldb + k), 0, -1, kBufferFlags);
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)(lds + i % D * STAGE);
#pragma unroll
        for (int j = 0; j < AL + BL; ++j) {
            const uint32_t m0reg = __builtin_amdgcn_readfirstlane(at + j * 1024);
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"(m0reg), "v"(off[j]), "s"(j < AL ? ra : rb)
                         : "memory");
        }
    };
    i32x4 acc[RT][2] = {};
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        if (d < n) send(d);
    for (int i = 0; i < n; ++i) {
        if (D == 2 || n - i < D - 1) wait_all_but<0>();
        else wait_all_but<(AL + BL) * (D - 2)>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last step's reads: their buffer is filled anew
        if (i + D - 1 < n) send(i + D - 1);
        const int8_t *const buf = lds + i % D * STAGE;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            i32x4 fa[RT], fb[2];
#pragma unroll
            for (int t = 0; t < RT; ++t)
                fa[t] = *(const i32x4 *)(buf + lds_unit<int8_t, true, false, 16>(t * 16 + (lane & 15), kk * 4 + (lane >> 4)));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fb[j] = *(const i32x4 *)(buf + AROWS * 128 +
                                         lds_unit<int8_t, true, true, 16>(row_of<true>(lane & 15, j), kk * 4 + (lane >> 4)));
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[t][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[t], acc[t][j], 0, 0, 0);
        }
    }
    const int t = wave, m = m0 + t * 16 + (lane & 15), c = n0 + (lane >> 4) * 8;  // a wave ends a tile of rows
    typename EPI::Column column;
    typename EPI::Item item;
    if (t < RT) {
        column = epi.template column<false>(c);
        item = epi.template item<false>(m, c);
    }
    __syncthreads();
    i32x4 *const red = (i32x4 *)smem;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) red[((wave * RT + r) * 2 + j) * 64 + lane] = acc[r][j];
    __syncthreads();
    if (t >= RT) return;
    Vec<float, 8> v;
    i32x4 sum[2] = {};
#pragma unroll
    for (int w = 0; w < kThinWaves; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) sum[j] += red[((w * RT + t) * 2 + j) * 64 + lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v.v[e] = (float)sum[0][e], v.v[4 + e] = (float)sum[1][e];
    epi.with([&](auto act) {
        epi.template store<decltype(act)::value, false>(m, c, v, (a.N + kThinCols - 1) / kThinCols * kThinCols, column, item);
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

    template <int RT>
    void thin() const {
        const int blocks = ((g.M + RT * 16 - 1) / (RT * 16)) * ((g.N + kThinCols - 1) / kThinCols);
        const auto kernel = k_q8_thin<RT, EpiQ8<YT>>;
        if constexpr (thin_lds(RT) > 65536)
            (void)hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, thin_lds(RT));
        hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(kThinWaves * 64), thin_lds(RT), st, args(), epi(), blocks);
    }

    void run() const {
        if (g.f.tile >= 0) return pick_q8_tile(g.f.tile, *this);
        if (g.f.tile == kQ8Thin) return g.M <= 16 ? thin<1>() : thin<2>();
        if (g.M == 1) few<1>();
        else few<2>();
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
