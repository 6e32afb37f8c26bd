// Backward of the product of codes.
//   dz = dy act'(z);  dx = (dz sw) wq;  dw = (dz sx)^T xq;  dbias = sum over the rows of dz
// Both products run on the int8 matrix cores: their left operands become whole
// numbers in fixed point of the largest magnitude of their row (column), in 8-bit
// digits, the right ones are the codes that the forward kept. The scales sw and
// sx, which belong to the summed index, are taken into dz before that.
//
// One kernel finds the largest magnitudes and the column sums, and transposes
// the codes, so that every operand has its summed index contiguous. A second
// writes the digits, of dz sx transposed. A third runs both products and the
// column sums' join side by side; a last one joins products that are split along
// k. dz is formed twice rather than kept: 3 bytes a value are read again where 4
// would be written and read.
//
// Four digits, whatever type the results have: a scale serves a whole row (for dw a
// column over all tokens), and what one loud token leaves the others of 16 bits is
// less than bf16 keeps. 2048 tokens, one with a gradient 10^4 times the others': dw is
// off by 10 % in norm where that token's code is 0 with two digits, by bf16's own
// 0.17 % with four. A plan may ask for two digits (round_dz). 8192 x 640 x 2560 bf16
// with gelu and z in codes takes 229 us with four, 30 + 71 + 143 + 8 in the trace, and
// 130 with two, 28 + 45 + 75: the first two kernels are bound by gelu's slope and by
// the loads' latency (2.3 and 3.3 TB/s), the third by the matrix cores
// (1500 TOPS in tiles of 128 x 128, 1430 with two digits). In fp32 1001 x 333 x 515
// takes 6.6 + 7.9 + 10.9.
#include "wq8_q8_gemm.h"
#include "wq8_rows.h"

namespace wq8 {
namespace {

enum { kZNone, kZValues, kZCodes };  // what the forward kept of z

// gelu's slope for bf16 results, Phi(z) + z phi(z), from that at -|z|, Phi(-|z|) - |z|
// phi(z), of which it is what is left of 1 for z >= 0. Phi(-|z|) as normal_cdf<false>()
// has it (1.5e-7), its half taken into the coefficients. 16 operations for 25: the
// slope is formed in both passes, and they are bound by that. Neither term is near
// 1/2, so the negative tail keeps three digits; as a difference from 1/2 it was off by
// 6 % at -5.5.
__device__ __forceinline__ float gelu_slope(float z) {
    const float a = fabsf(z), e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);  // exp(-z^2 / 2)
    const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752f, a, 1.0f));
    float s = fmaf(0.5307027145f, t, -0.7265760135f);
    s = fmaf(s, t, 0.7107068705f);
    s = fmaf(s, t, -0.142248368f);
    s = fmaf(s, t, 0.127414796f);
    const float low = fmaf(a * -0.3989422804014327f, e, s * t * e);
    return z < 0.0f ? low : 1.0f - low;
}

template <int ACT, bool EXACT>
__device__ __forceinline__ float slope_of(float z) {
    if constexpr (ACT == WQ8_ACT_GELU && !EXACT) return gelu_slope(z);
    return act_slope<ACT, EXACT>(z);
}

// What dz of V columns of a row is made of, and dz: zeros past the last column (a
// group of z's codes that stands for NaN has columns before it as well, and makes
// the row's products NaN).
template <typename YT, int ZF, int V = kV>
struct DzParts {
    using Codes = std::conditional_t<V == 8, uint64_t, uint32_t>;
    Vec<YT, V> dy, z;
    Codes codes;
    float scale;

    __device__ __forceinline__ static Vec<YT, V> some(const YT *row, int c, int C) {
        if constexpr (V == kV) return load_any<YT>(row, c, C);
        else return load_vec_n<YT, V>(row + c, C - c);
    }
    // WHOLE: all columns exist.
    template <bool WHOLE>
    __device__ __forceinline__ void load(const Q8Geo &g, const Q8Ptrs &a, int64_t row, int c) {
        if constexpr (WHOLE) dy = load_vec<YT, V>((const YT *)a.dy + row * g.ys + c);
        else dy = some((const YT *)a.dy + row * g.ys, c, g.N);
        if constexpr (ZF == kZValues) {
            if constexpr (WHOLE) z = load_vec<YT, V>((const YT *)a.z_in + row * g.N + c);
            else z = some((const YT *)a.z_in + row * g.N, c, g.N);
        }
        if constexpr (ZF == kZCodes) {
            codes = *(const Codes *)(a.zq_in + row * g.Np + min(c, g.Np - V));
            scale = a.sz_in[row * ((g.N + 31) / 32) + min(c, g.N - 1) / 32];
        }
    }
    template <int ACT, bool EXACT>
    __device__ __forceinline__ void form(float (&dz)[V]) const {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dz[k] = to_f32(dy.v[k]);
            if constexpr (ACT != WQ8_ACT_NONE) {
                float v;
                // code scale, rounded once, from code + 128: unsigned bytes convert in one step
                if constexpr (ZF == kZCodes)
                    v = fmaf((float)(uint8_t)((codes ^ (Codes)0x8080808080808080ull) >> (8 * k)), scale, -128.0f * scale);
                else v = to_f32(z.v[k]);
                dz[k] *= slope_of<ACT, EXACT>(v);
            }
        }
    }
};

// ------------------------------------------------------------------ first pass
// 64 lanes x 8 columns of `chunk` rows, a wave each: the largest |dz sw| of every
// row, the largest |dz sx| and the sum of dz of every column.
// Eight waves a block: the second pass reads what each block has found.
constexpr int kMaxCols = 64 * kV;
constexpr int kMaxRows = 2;  // rows of a wave whose loads are in flight together
constexpr int kMaxWaves = 8;

template <typename XT, typename YT, int ZF>
__device__ __forceinline__ void max_block(const Q8Geo &g, const Q8Ptrs &a, int b) {
    __shared__ float red[kMaxWaves - 1][2][kMaxCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int chunk = b / g.ncol, col = b - chunk * g.ncol;
    const int c = col * kMaxCols + lane * kV;
    const int r0 = chunk * g.chunk, r1 = min(r0 + g.chunk, g.M);
    const Vec<float, kV> sw = load_any<float>(a.sw, c, g.N);
    float sum[kV] = {}, most[kV] = {};
    with_act(g.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        if constexpr ((A == WQ8_ACT_NONE) == (ZF == kZNone))
        {
            const auto rows = [&](auto whole) {
                for (int r = r0 + wave; r < r1; r += kMaxWaves * kMaxRows) {
                    DzParts<YT, ZF> parts[kMaxRows];
                    float dz[kMaxRows][kV], sx[kMaxRows];
#pragma unroll
                    for (int i = 0; i < kMaxRows; ++i) {
                        const int row = min(r + kMaxWaves * i, r1 - 1);
                        parts[i].template load<decltype(whole)::value>(g, a, row, c);
                        sx[i] = a.sx[row];
                    }
#pragma unroll
                    for (int i = 0; i < kMaxRows; ++i) parts[i].template form<A, exact_acts<XT, YT>()>(dz[i]);
#pragma unroll
                    for (int i = 0; i < kMaxRows; ++i)
                        if (r + kMaxWaves * i < r1) {
                            float m = 0.0f;
#pragma unroll
                            for (int k = 0; k < kV; ++k) {
                                m = larger(m, dz[i][k] * sw.v[k]);
                                most[k] = larger(most[k], dz[i][k] * sx[i]);
                                sum[k] += dz[i][k];
                            }
                            const uint32_t top = wave_max(bits_of(m));
                            if (lane == 0) a.rowmax[(int64_t)col * g.M + r + kMaxWaves * i] = __uint_as_float(top);
                        }
                }
            };
            if ((col + 1) * kMaxCols <= g.N) rows(std::true_type{});
            else rows(std::false_type{});
        }
    });
    if (wave > 0)
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            red[wave - 1][0][k * 64 + lane] = most[k];
            red[wave - 1][1][k * 64 + lane] = sum[k];
        }
    __syncthreads();
    if (wave > 0 || c >= g.Np) return;
    Vec<float, kV> m, s;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
        m.v[k] = most[k];
        s.v[k] = sum[k];
#pragma unroll
        for (int w = 0; w < kMaxWaves - 1; ++w) {
            m.v[k] = larger(m.v[k], red[w][0][k * 64 + lane]);
            s.v[k] += red[w][1][k * 64 + lane];
        }
    }
    store_vec<float, kV>(a.colmax + (int64_t)chunk * g.Np + c, m);
    store_vec<float, kV>(a.colsum + (int64_t)chunk * g.Np + c, s);
}

// The p-th bytes, from the top of N bytes, of four numbers: out[p].
template <int N>
__device__ __forceinline__ void bytes_of(const uint32_t (&q)[4], uint32_t (&out)[N]) {
    const auto pick = [](uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); };
    const uint32_t a = pick(q[1], q[0], 0x05010400u), b = pick(q[3], q[2], 0x05010400u);  // bytes 0, then 1, of both
    out[N - 1] = pick(b, a, 0x05040100u);
    out[N - 2] = pick(b, a, 0x07060302u);
    if constexpr (N == 4) {
        const uint32_t c = pick(q[1], q[0], 0x07030602u), d = pick(q[3], q[2], 0x07030602u);
        out[1] = pick(d, c, 0x05040100u);
        out[0] = pick(d, c, 0x07060302u);
    }
}

// A matrix of codes [rows][ld] transposed to [cols][tld], zeros behind its last
// row: 128 x 128 codes a block. A thread has 4 rows of 8 columns.
__device__ __forceinline__ void transpose_block(const int8_t *x, int64_t rows, int cols, int64_t ld, int8_t *t, int64_t tld, int b) {
    constexpr int LD = 128 + 4;  // bytes between columns in LDS
    __shared__ __align__(16) int8_t tile[128 * LD];
    const int across = (int)(ld / 128);
    const int64_t r0 = (int64_t)(b / across) * 128;
    const int c0 = (b - b / across * across) * 128;
    const int rg = threadIdx.x >> 4, cg = threadIdx.x & 15;
    uint32_t v[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + rg * 4 + i;
        const uint64_t q = *(const uint64_t *)(x + min(r, rows - 1) * ld + c0 + cg * 8);
        v[i][0] = r < rows ? (uint32_t)q : 0u;
        v[i][1] = r < rows ? (uint32_t)(q >> 32) : 0u;
    }
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const uint32_t rows4[4] = {v[0][d], v[1][d], v[2][d], v[3][d]};
        uint32_t o[4];
        bytes_of<4>(rows4, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) *(uint32_t *)(tile + (cg * 8 + d * 4 + e) * LD + rg * 4) = o[3 - e];
    }
    __syncthreads();
    // a wave writes 8 columns' lines of 128 bytes at a time, 16 bytes a lane
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = i * 64 + (threadIdx.x >> 3), part = (threadIdx.x & 7) * 16;
        v4i o;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = *(const int *)(tile + col * LD + part + d * 4);
        if (c0 + col < cols) *(v4i *)(t + (int64_t)(c0 + col) * tld + r0 + part) = o;
    }
}

// Blocks [0, nm): largest magnitudes; then nx of xq's transposition and the rest of wq's.
template <typename XT, typename YT, int ZF>
__global__ __launch_bounds__(kMaxWaves * 64) void k_q8_max(Q8Geo g, Q8Ptrs a, int nm, int nx, int nb) {
    int b;
    if (!block_number(nb, b)) return;
    if (b < nm) max_block<XT, YT, ZF>(g, a, b);
    else if (b < nm + nx) transpose_block(a.xq, g.M, g.K, g.Kp, a.xt, g.Mp, b - nm);
    else transpose_block(a.wq, g.N, g.K, g.Kp, a.wt, g.Np, b - nm - nx);
}

// ----------------------------------------------------------------- second pass
// Fixed point of a largest magnitude m (its bits): whole numbers of `planes` digits, the
// highest in [-127, 127], the others in [-128, 127]. An infinity or a NaN: a scale of
// NaN, and any digits.
template <int PLANES>
struct Digits {
    static constexpr float kMost = PLANES == 2 ? 32512.0f : 2130706432.0f;  // 127 256^(planes - 1)
    float f, up;  // found once a row or column, and read from LDS

    __device__ __forceinline__ void find(uint32_t bits) {
        const float m = __uint_as_float(bits);
        up = m < 0x1p-60f ? 0x1p64f : 1.0f;  // kMost / m overflows below 2^-96
        f = bits == 0 || bits >= kInfBits ? 0.0f : kMost / (m * up);
    }
    // What a sum of products has to be multiplied by, in units of the highest digit.
    __device__ __forceinline__ static float scale(uint32_t bits) {
        return bits >= kInfBits ? __uint_as_float(0x7fc00000u) : __uint_as_float(bits) / 127.0f;
    }
    // The number plus 128 in each digit but the highest: its bytes, with 128 taken
    // off again in each by lower(), are the digits.
    __device__ __forceinline__ uint32_t operator()(float v) const {
        if constexpr (PLANES == 2) return __float_as_uint(fmaf(v, f, kRoundMagic + 128.0f));  // the low half
        // 2130706432 (1 + 2^-23) + 0x808080 is still below 2^31
        return (uint32_t)(int)__builtin_rintf(v * f) + 0x00808080u;
    }
    __device__ __forceinline__ static void lower(uint32_t (&planes)[PLANES]) {
#pragma unroll
        for (int p = 1; p < PLANES; ++p) planes[p] ^= 0x80808080u;
    }
};

// 128 rows x 32 columns: a thread has 4 rows of 4 columns. With 8 columns it has
// fewer and longer waves: 1024 x 640 x 640 then takes 22.2 us for 20.0 with two digits
// and 33.1 for 29.3 with four, 8192 x 640 x 2560 130.3 for 128.5 and 238 for 248.
template <typename XT, typename YT, int ZF, int PLANES>
__global__ __launch_bounds__(256) void k_q8_digits(Q8Geo g, Q8Ptrs a, int want_dx, int want_dw, int nb) {
    constexpr int V = 4, COLS = 8 * V, ACROSS = COLS / 4, ALONG = 256 / ACROSS;
    constexpr int LD = 128 + 4;  // bytes between columns in LDS: a wave's stores meet every bank twice
    __shared__ __align__(16) int8_t tile[PLANES * COLS * LD];
    __shared__ float cpart[ALONG][COLS];
    __shared__ Digits<PLANES> cdig[COLS], rdig[128];
    int b;
    if (!block_number(nb, b)) return;
    b = xcd_block(b, nb);  // blocks that share lines of z's codes and of the rows' digits behind one cache
    const int across = g.Np / COLS, br = b / across, r0 = br * 128, c0 = (b - br * across) * COLS;
    const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3, c = c0 + cg * V;
    DzParts<YT, ZF, V> parts[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = min(r0 + rg * 4 + i, g.M - 1);
        if (c0 + COLS <= g.N) parts[i].template load<true>(g, a, r, c);
        else parts[i].template load<false>(g, a, r, c);
    }
    if (want_dw) {  // 4 columns a thread, the others along the first pass's chunks
        const int c4 = (threadIdx.x % ACROSS) * 4, q = threadIdx.x / ACROSS;
        Vec<float, 4> m = {};
#pragma unroll 8
        for (int i = q; i < g.nchunk; i += ALONG) {
            const Vec<float, 4> v = load_vec<float, 4>(a.colmax + (int64_t)i * g.Np + c0 + c4);
#pragma unroll
            for (int k = 0; k < 4; ++k) m.v[k] = larger(m.v[k], v.v[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) cpart[q][c4 + k] = m.v[k];
    }
    if (want_dx && threadIdx.x < 128) {
        const int r = min(r0 + (int)threadIdx.x, g.M - 1);
        float m = 0.0f;
        for (int i = 0; i < g.ncol; ++i) m = larger(m, a.rowmax[(int64_t)i * g.M + r]);
        rdig[threadIdx.x].find(bits_of(m));
        if (c0 == 0 && r0 + (int)threadIdx.x < g.M) a.rscale[r] = Digits<PLANES>::scale(bits_of(m));
    }
    float dz[4][V];
    with_act(g.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        if constexpr ((A == WQ8_ACT_NONE) == (ZF == kZNone))
#pragma unroll
            for (int i = 0; i < 4; ++i) parts[i].template form<A, exact_acts<XT, YT>()>(dz[i]);
    });
    __syncthreads();
    if (want_dw && threadIdx.x < COLS) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < ALONG; ++i) t = larger(t, cpart[i][threadIdx.x]);
        cdig[threadIdx.x].find(bits_of(t));
        if (br == 0 && c0 + (int)threadIdx.x < g.N) a.cscale[c0 + threadIdx.x] = Digits<PLANES>::scale(bits_of(t));
    }
    if (want_dx) {
        const Vec<float, V> sw = load_vec_n<float, V>(a.sw + c, g.N - c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + rg * 4 + i;
            const Digits<PLANES> d = rdig[rg * 4 + i];
            float u[V];
#pragma unroll
            for (int k = 0; k < V; ++k) u[k] = dz[i][k] * sw.v[k];
            if (__builtin_expect(__any(d.up != 1.0f), 0))
#pragma unroll
                for (int k = 0; k < V; ++k) u[k] *= d.up;
            uint32_t o[PLANES];
            bytes_of<PLANES>({d(u[0]), d(u[1]), d(u[2]), d(u[3])}, o);
            Digits<PLANES>::lower(o);
            if (r < g.M)
#pragma unroll
                for (int p = 0; p < PLANES; ++p) *(uint32_t *)(a.ur + ((int64_t)p * g.M + r) * g.Np + c) = o[p];
        }
    }
    if (!want_dw) return;
    __syncthreads();
    float sx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sx[i] = r0 + rg * 4 + i < g.M ? a.sx[r0 + rg * 4 + i] : 0.0f;  // past the end dz is the last row's
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const Digits<PLANES> d = cdig[cg * V + k];
        float u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = dz[i][k] * sx[i];
        if (__builtin_expect(__any(d.up != 1.0f), 0))
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] *= d.up;
        uint32_t o[PLANES];
        bytes_of<PLANES>({d(u[0]), d(u[1]), d(u[2]), d(u[3])}, o);
        Digits<PLANES>::lower(o);
#pragma unroll
        for (int p = 0; p < PLANES; ++p) *(uint32_t *)(tile + (p * COLS + cg * V + k) * LD + rg * 4) = o[p];
    }
    __syncthreads();
    // 8 bytes a lane, 16 lanes a line
#pragma unroll
    for (int i = 0; i < PLANES * COLS / 16; ++i) {
        const int line = i * 16 + (threadIdx.x >> 4), p = line / COLS, col = line % COLS, part = (threadIdx.x & 15) * 8;
        const uint32_t *const from = (const uint32_t *)(tile + line * LD + part);
        if (c0 + col < g.N)
            *(uint64_t *)(a.uc + ((int64_t)p * g.N + c0 + col) * g.Mp + r0 + part) = (uint64_t)from[1] << 32 | from[0];
    }
}

// ---------------------------------------------------------------- the products
template <typename T, int PLANES>
struct EpiScale {
    T *out;
    int64_t ld;
    int M, N;
    const float *scale;  // of the rows

    struct Column {};
    struct Item {
        float scale;
    };
    __device__ __forceinline__ bool plain() const { return true; }
    template <bool>
    __device__ __forceinline__ Column column(int) const { return {}; }
    template <bool>
    __device__ __forceinline__ Item item(int m, int) const { return {scale[min(m, M - 1)]}; }
    template <typename F>
    __device__ __forceinline__ void with(F f) const {
        f(std::integral_constant<int, WQ8_ACT_NONE>{});
    }

    template <int ACT, bool WHOLE>
    __device__ __forceinline__ void store(int m, int n, const Vec<float, 8> &v, int, Column, const Item &item) const {
        if (!WHOLE && (m >= M || n >= N)) return;
        Vec<T, 8> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(v.v[e] * (PLANES == 2 ? 0x1p-8f : 0x1p-16f) * item.scale);
        if constexpr (WHOLE) store_vec<T, 8>(out + (int64_t)m * ld + n, r);
        else store_vec_n<T, 8>(out + (int64_t)m * ld + n, r, N - n);
    }
};

// dbias: the chunks' column sums, 16 columns a block, its other threads along the chunks.
__device__ __forceinline__ void dbias_block(const Q8Geo &g, const Q8Ptrs &a, int b) {
    extern __shared__ __align__(128) char smem[];
    float *red = (float *)smem;
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, rows = blockDim.x >> 4, c = b * 16 + tc;
    float t = 0.0f;
    if (c < g.N)
        for (int r = tr; r < g.nchunk; r += rows) t += a.colsum[(int64_t)r * g.Np + c];
    red[tr * 17 + tc] = t;
    __syncthreads();
    if (tr == 0 && c < g.N) {
        float s = 0.0f;
        for (int i = 0; i < rows; ++i) s += red[i * 17 + tc];
        a.dbias[c] = s;
    }
}

// Blocks [0, nw): dw; [nw, nw + nx): dx; the rest: dbias.
template <typename T, int PLANES, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN * 64) void k_q8_bwd(Q8Args dw, EpiScale<T, PLANES> ew, int nw, Q8Args dx, EpiScale<T, PLANES> ex,
                                                        int nx, int nb, Q8Geo g, Q8Ptrs p) {
    int b;
    if (!block_number(nb, b)) return;
    if (b < nw + nx) {  // one copy of the product: which one is the same for a whole block
        const bool first = b < nw;
        const Q8Args q = first ? dw : dx;
        const EpiScale<T, PLANES> e = first ? ew : ex;
        q8_block<BM, BN, WM, WN, PLANES>(q, e, first ? b : b - nw, first ? nw : nx);
    } else {
        dbias_block(g, p, b - nw - nx);
    }
}

template <typename T, int PLANES>
__global__ __launch_bounds__(256) void k_q8_bwd_join(Q8Args dw, EpiScale<T, PLANES> ew, int nw, Q8Args dx, EpiScale<T, PLANES> ex,
                                                     int nb) {
    int b;
    if (!block_number(nb, b)) return;
    if (b < nw) q8_join_block<PLANES>(dw, ew, b);
    else q8_join_block<PLANES>(dx, ex, b - nw);
}

template <typename T>
__global__ __launch_bounds__(256) void k_q8_zero(T *dw, int64_t values, float *dbias, int N) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; dw && i < values; i += step) dw[i] = T(0);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; dbias && i < N; i += step) dbias[i] = 0.0f;
}

template <typename T, int PLANES>
struct RunQ8Backward {
    const Q8Geo &g;
    const Q8Ptrs &p;
    hipStream_t st;

    template <int BM, int BN, int WM, int WN>
    void operator()() const {
        Q8Args dw = {}, dx = {};
        int64_t nw = 0, nx = 0, jw = 0, jx = 0;
        if (p.dw) {
            dw.A = p.uc;
            dw.B = p.xt;
            dw.lda = dw.ldb = g.Mp;
            dw.M = g.N;
            dw.N = g.K;
            dw.steps = g.Mp / 128;
            dw.plane = (int64_t)g.N * g.Mp;
            nw = q8_tiles<BM, BN>(dw, g.dw, p.partial_dw);
            jw = q8_join_blocks(dw);
        }
        if (p.dx) {
            dx.A = p.ur;
            dx.B = p.wt;
            dx.lda = dx.ldb = g.Np;
            dx.M = g.M;
            dx.N = g.K;
            dx.steps = g.Np / 128;
            dx.plane = (int64_t)g.M * g.Np;
            nx = q8_tiles<BM, BN>(dx, g.dx, p.partial_dx);
            jx = q8_join_blocks(dx);
        }
        const EpiScale<T, PLANES> ew = {(T *)p.dw, g.K, g.N, g.K, p.cscale}, ex = {(T *)p.dx, g.xs, g.M, g.K, p.rscale};
        const int64_t blocks = nw + nx + (p.dbias ? (g.N + 15) / 16 : 0);
        if (blocks > 0) {
            const auto kernel = k_q8_bwd<T, PLANES, BM, BN, WM, WN>;
            hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(WM * WN * 64), (q8_lds<BM, BN, PLANES>(kernel)), st, dw, ew, (int)nw, dx, ex,
                               (int)nx, (int)blocks, g, p);
        }
        if (jw + jx > 0)
            hipLaunchKernelGGL((k_q8_bwd_join<T, PLANES>), grid_of(jw + jx), dim3(256), 0, st, dw, ew, (int)jw, dx, ex, (int)(jw + jx));
    }
};

template <typename XT, typename YT, int ZF, int PLANES>
void prepare(const Q8Geo &g, const Q8Ptrs &p, hipStream_t st) {
    const auto tiles = [](int64_t rows, int64_t bytes) { return (rows + 127) / 128 * (bytes / 128); };
    const int64_t nm = (int64_t)g.nchunk * g.ncol, nx = p.dw ? tiles(g.M, g.Kp) : 0, nw = p.dx ? tiles(g.N, g.Kp) : 0;
    hipLaunchKernelGGL((k_q8_max<XT, YT, ZF>), grid_of(nm + nx + nw), dim3(kMaxWaves * 64), 0, st, g, p, (int)nm, (int)nx,
                       (int)(nm + nx + nw));
    if (!p.dx && !p.dw) return;
    const int64_t nd = (int64_t)(g.Mp / 128) * (g.Np / 32);
    hipLaunchKernelGGL((k_q8_digits<XT, YT, ZF, PLANES>), grid_of(nd), dim3(256), 0, st, g, p, p.dx != nullptr, p.dw != nullptr,
                       (int)nd);
}

template <typename XT, typename YT, int PLANES>
void products(const Q8Geo &g, const Q8Ptrs &p, hipStream_t st) {
    if (g.act == WQ8_ACT_NONE) prepare<XT, YT, kZNone, PLANES>(g, p, st);
    else if (p.z_in) prepare<XT, YT, kZValues, PLANES>(g, p, st);
    else prepare<XT, YT, kZCodes, PLANES>(g, p, st);
    pick_q8_pair_tile(g.dw.tile, RunQ8Backward<XT, PLANES>{g, p, st});
}

template <typename XT, typename YT>
void backward(const Q8Geo &g, const Q8Ptrs &p, hipStream_t st) {
    if (g.M == 0) {
        if (p.dw || p.dbias)
            hipLaunchKernelGGL(k_q8_zero<XT>, dim3(256), dim3(256), 0, st, (XT *)p.dw, (int64_t)g.N * g.K, p.dbias, g.N);
        return;
    }
    if (!p.dx && !p.dw && !p.dbias) return;
    if constexpr (sizeof(XT) == 2)
        if (g.planes == 2) return products<XT, YT, 2>(g, p, st);
    products<XT, YT, 4>(g, p, st);
}

}  // namespace

wq8_status launch_q8_backward(const Q8Geo &g, wq8_dtype xdt, wq8_dtype ydt, const Q8Ptrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (xdt == WQ8_F32) {
        if (ydt == WQ8_F32) backward<float, float>(g, p, st);
        else backward<float, bf16_t>(g, p, st);
    } else {
        if (ydt == WQ8_F32) backward<bf16_t, float>(g, p, st);
        else backward<bf16_t, bf16_t>(g, p, st);
    }
    return check_launch("backward of the product of codes");
}

}  // namespace wq8
