// Backward of the matrix product with bias, activation and residual.
//   dz = dy act'(z);  dx = dz w;  dw = dz^T x;  dbias = sum over the rows of dz
// One kernel forms dz (once, for the products) with the column sums of its fp32
// values. A second one runs both products and the column sums' join side by
// side: they only share inputs, and the blocks of one fill the compute units
// that the other leaves idle. The products read dz, w and x as they lie: the
// operand whose row index is contiguous goes through the transposing LDS
// reads, so nothing is transposed in memory. A last kernel joins the sums of
// products that are split along k.
//
// For bf16 products dz is held as two matrices of their type that are
// multiplied one after the other, k step by k step (dbias sums fp32 values).
// Rounded to bf16 once, as a caller may ask for, it adds as much error to dx
// and dw as their own final rounding, sqrt 2 times the error of one rounding,
// over few values and over many.
// Measured: 8192 x 640 x 2560 bf16 with gelu 187 to 192 us: dz 34 us (168 MB, 4.9
// TB/s, bound by memory), the products 151 us (both halves of dz: 107 GFLOP, 710
// TFLOP/s) and the join 7 us. With dz rounded once 117 to 121 us: 26, 84 and 7.
// 16384 x 2560 x 10240 with gelu 3.58 ms, rounded 1.82 ms (946 TFLOP/s, in 256 x
// 256 tiles, though these spill 31 registers); 1001 x 333 x 515 fp32, rows at odd addresses, 23 us in kernels of
// 4, 16 and 4 us, bound by launches and load latency. One kernel for both
// products instead of two, a join each and one for dbias: 127 and 36 us before.
#include "wq8_gemm_device.h"

namespace wq8 {
namespace {

// dz of 64 x V columns (a wave per row, kDzRows rows in flight) over `chunk` rows,
// and their sums. A vector that would pass the last column starts earlier: its
// first `lo` values are another thread's, stored twice and summed once.
constexpr int kDzRows = 4;

// v as the sum of two bf16 values: its first 8 bits, cut off, and what that
// leaves, rounded: within 2^-16 of v. Where nothing is left the first is the
// next number towards zero and the second the difference, exactly. So both
// have v's sign and neither is zero unless v is: an infinity that they are
// multiplied by gives the same infinity twice, where a zero or another sign
// would make it a NaN. (A smallest number in place of the zero is not the same:
// the matrix cores drop a unit in the last place of a sum that it is taken from.)
__device__ __forceinline__ void split_dz(float v, bf16_t &top, bf16_t &rest) {
    const uint32_t u = __float_as_uint(v);
    bf16_t t = (bf16_t)(u >> 16);
    if (fabsf(v - to_f32(t)) < 0x1p-126f && (t & 0x7fff)) --t;
    top = t;
    rest = from_f32<bf16_t>(v - to_f32(t));
    if (!(fabsf(v) < INFINITY)) top = rest = from_f32<bf16_t>(v);
}

template <typename XT, typename YT, int V>
__global__ __launch_bounds__(256) void k_dz(LinearGeo g, LinearPtrs a, int ncol, int want_sum) {
    __shared__ float red[3][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int b;
    if (!block_number(ncol * g.dz_nchunk, b)) return;
    const int chunk = b / ncol;
    const int c = ((b - chunk * ncol) * 64 + lane) * V, n = min(c, g.N - V), lo = min(c - n, V);
    const int r0 = chunk * g.dz_chunk, r1 = min(r0 + g.dz_chunk, g.M);
    const YT *dy = (const YT *)a.dy, *z = (const YT *)a.zin;
    XT *dz = (XT *)a.dz;
    float sum[V] = {};
    with_act(g.act, [&](auto act) {
        constexpr int A = decltype(act)::value;
        for (int r = r0 + wave; r < r1; r += 4 * kDzRows) {
            Vec<YT, V> d[kDzRows], zz[kDzRows];
#pragma unroll
            for (int i = 0; i < kDzRows; ++i) {
                const int64_t row = min(r + 4 * i, r1 - 1);
                d[i] = load_vec<YT, V>(dy + row * g.ys + n);
                if constexpr (A != WQ8_ACT_NONE) zz[i] = load_vec<YT, V>(z + row * g.N + n);
            }
#pragma unroll
            for (int i = 0; i < kDzRows; ++i)
                if (r + 4 * i < r1) {
                    Vec<XT, V> o, rest;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        float v = to_f32(d[i].v[k]);
                        if constexpr (A != WQ8_ACT_NONE) v *= act_slope<A, exact_acts<XT, YT>()>(to_f32(zz[i].v[k]));
                        sum[k] += v;
                        if constexpr (sizeof(XT) == 2) split_dz(v, o.v[k], rest.v[k]);
                        if (sizeof(XT) == 4 || g.dz_planes == 1) o.v[k] = from_f32<XT>(v);
                    }
                    if (dz && lo < V) {
                        XT *const to = dz + (int64_t)(r + 4 * i) * g.N + n;
                        store_vec<XT, V>(to, o);
                        if (sizeof(XT) == 2 && g.dz_planes == 2) store_vec<XT, V>(to + (int64_t)g.M * g.N, rest);
                    }
                }
        }
    });
    if (!want_sum) return;
    if (wave > 0)
#pragma unroll
        for (int k = 0; k < V; ++k) red[wave - 1][lane * V + k] = sum[k];
    __syncthreads();
    if (wave == 0)
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k >= lo)
                a.colsum[(int64_t)chunk * g.N + n + k] =
                    (sum[k] + red[0][lane * V + k]) + (red[1][lane * V + k] + red[2][lane * V + k]);
}

// dbias: the chunks' column sums, 16 columns a block, its other threads along
// the chunks.
__device__ __forceinline__ void dbias_block(const LinearGeo &g, const LinearPtrs &a, int b) {
    extern __shared__ __align__(128) char smem[];
    float *red = (float *)smem;
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, rows = blockDim.x >> 4, c = b * 16 + tc;
    float t = 0.0f;
    if (c < g.N)
        for (int r = tr; r < g.dz_nchunk; r += rows) t += a.colsum[(int64_t)r * g.N + c];
    red[tr * 17 + tc] = t;
    __syncthreads();
    if (tr == 0 && c < g.N) {
        float s = 0.0f;
        for (int i = 0; i < rows; ++i) s += red[i * 17 + tc];
        a.dbias[c] = s;
    }
}

template <typename T>
struct EpiStore {
    T *out;
    int64_t ld;

    struct Column {};
    struct Item {};
    __device__ __forceinline__ Column column(int) const { return {}; }
    __device__ __forceinline__ Item item(int, int) const { return {}; }
    template <typename F>
    __device__ __forceinline__ void with(F f) const {
        f(std::integral_constant<int, WQ8_ACT_NONE>{});
    }

    template <int ACT>
    __device__ __forceinline__ void store(int m, int n, const Vec<float, 8> &v, int cnt, Column, Item) const {
        Vec<T, 8> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(v.v[e]);
        store_vec_n<T, 8>(out + (int64_t)m * ld + n, r, cnt);
    }
};

// Blocks [0, nw): dw; [nw, nw + nx): dx; the rest: dbias.
template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM *WN * 64) void k_linear_bwd(GemmArgs dw, EpiStore<T> ew, int nw, GemmArgs dx, EpiStore<T> ex,
                                                            int nx, int nb, LinearGeo g, LinearPtrs p) {
    constexpr bool TWO = sizeof(T) == 2;
    int b;
    if (!block_number(nb, b)) return;
    if (b < nw) gemm_block<T, false, false, BM, BN, WM, WN, DIRECT, TWO>(dw, ew, b, nw);
    else if (b < nw + nx) gemm_block<T, true, false, BM, BN, WM, WN, DIRECT, TWO>(dx, ex, b - nw, nx);
    else dbias_block(g, p, b - nw - nx);
}

template <typename T>
__global__ __launch_bounds__(256) void k_linear_bwd_join(GemmArgs dw, EpiStore<T> ew, int nw, GemmArgs dx, EpiStore<T> ex,
                                                         int nb) {
    int b;
    if (!block_number(nb, b)) return;
    if (b < nw) join_block(dw, ew, b);
    else join_block(dx, ex, b - nw);
}

template <typename T>
struct RunBackward {
    const LinearGeo &g;
    const LinearPtrs &p;
    hipStream_t st;

    template <int BM, int BN, int WM, int WN, bool DIRECT>
    void operator()() const {
        const void *dz = g.dz_own ? p.dz : p.dy;
        const int64_t ldz = g.dz_own ? g.N : g.ys;
        GemmArgs dw = {}, dx = {};
        int64_t nw = 0, nx = 0, jw = 0, jx = 0;
        if (p.dw) {
            dw.A = dz;
            dw.more = g.dz_planes - 1;
            dw.plane = (int64_t)g.M * g.N;
            dw.lda = ldz;
            dw.B = p.x;
            dw.ldb = g.xs;
            dw.M = g.N;
            dw.N = g.K;
            dw.K = g.M;
            nw = set_tiles<BM, BN>(dw, g.dw, p.partial_dw);
            jw = join_blocks(dw);
        }
        if (p.dx && g.M > 0) {
            dx.A = dz;
            dx.more = g.dz_planes - 1;
            dx.plane = (int64_t)g.M * g.N;
            dx.lda = ldz;
            dx.B = p.w;
            dx.ldb = g.K;
            dx.M = g.M;
            dx.N = g.K;
            dx.K = g.N;
            nx = set_tiles<BM, BN>(dx, g.dx, p.partial_dx);
            jx = join_blocks(dx);
        }
        const EpiStore<T> ew = {(T *)p.dw, g.K}, ex = {(T *)p.dx, g.xs};
        const int64_t blocks = nw + nx + (p.dbias ? (g.N + 15) / 16 : 0);
        if (blocks > 0) {
            const auto kernel = k_linear_bwd<T, BM, BN, WM, WN, DIRECT>;
            hipLaunchKernelGGL(kernel, grid_of(blocks), dim3(WM * WN * 64), (tile_lds<BM, BN>(kernel)), st, dw, ew, (int)nw, dx,
                               ex, (int)nx, (int)blocks, g, p);
        }
        if (jw + jx > 0)
            hipLaunchKernelGGL((k_linear_bwd_join<T>), grid_of(jw + jx), dim3(256), 0, st, dw, ew, (int)jw, dx, ex,
                               (int)(jw + jx));
    }
};

template <typename XT, typename YT>
void backward(const LinearGeo &g, const LinearPtrs &p, hipStream_t st) {
    constexpr int V = 16 / (sizeof(XT) > sizeof(YT) ? sizeof(XT) : sizeof(YT));
    if (g.M > 0 && (p.dbias || (g.dz_own && (p.dx || p.dw)))) {
        const auto go = [&](auto kernel, int v) {
            const int ncol = (g.N + 64 * v - 1) / (64 * v);
            hipLaunchKernelGGL(kernel, grid_of((int64_t)ncol * g.dz_nchunk), dim3(256), 0, st, g, p, ncol, p.dbias != nullptr);
        };
        if (g.N >= V) go(k_dz<XT, YT, V>, V);
        else go(k_dz<XT, YT, 1>, 1);
    }
    pick_tile<sizeof(XT) == 4>(g.dw, RunBackward<XT>{g, p, st});
}

}  // namespace

wq8_status launch_linear_backward(const LinearGeo &g, wq8_dtype xdt, wq8_dtype ydt, const LinearPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (xdt == WQ8_F32) {
        if (ydt == WQ8_F32) backward<float, float>(g, p, st);
        else backward<float, bf16_t>(g, p, st);
    } else {
        if (ydt == WQ8_F32) backward<bf16_t, float>(g, p, st);
        else backward<bf16_t, bf16_t>(g, p, st);
    }
    return check_launch("matrix product backward");
}

}  // namespace wq8
