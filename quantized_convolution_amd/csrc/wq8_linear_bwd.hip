// Backward of the matrix product with bias, activation and residual.
//   dz = dy act'(z);  dx = dz w;  dw = dz^T x;  dbias = sum over the rows of dz
// One kernel forms dz (once, in x's type) with the column sums of the unrounded
// values; dx and dw are tiled products that read dz, w and x as they lie: the
// operand whose row index is contiguous goes through the transposing LDS
// reads, so nothing is transposed in memory.
#include "wq8_gemm_device.h"

namespace wq8 {
namespace {

// dz of 64 x V columns (a wave per row, kDzRows rows in flight) over `chunk` rows,
// and their sums. A vector that would pass the last column starts earlier: its
// first `lo` values are another thread's, stored twice and summed once.
constexpr int kDzRows = 4;
template <typename XT, typename YT, int V>
__global__ __launch_bounds__(256) void k_dz(LinearGeo g, LinearPtrs a, int ncol, int want_sum) {
    __shared__ float red[3][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int chunk = blockIdx.x / ncol;
    const int c = ((blockIdx.x - chunk * ncol) * 64 + lane) * V, n = min(c, g.N - V), lo = min(c - n, V);
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
                    Vec<XT, V> o;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        float v = to_f32(d[i].v[k]);
                        if constexpr (A != WQ8_ACT_NONE) v *= act_slope<A>(to_f32(zz[i].v[k]));
                        sum[k] += v;
                        o.v[k] = from_f32<XT>(v);
                    }
                    if (dz && lo < V) store_vec<XT, V>(dz + (int64_t)(r + 4 * i) * g.N + n, o);
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

// dbias: the chunks' column sums, 16 columns x 16 lanes along the chunks.
__global__ __launch_bounds__(256) void k_dbias(LinearGeo g, LinearPtrs a) {
    __shared__ float red[16][17];
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, c = blockIdx.x * 16 + tc;
    float t = 0.0f;
    if (c < g.N)
        for (int r = tr; r < g.dz_nchunk; r += 16) t += a.colsum[(int64_t)r * g.N + c];
    red[tr][tc] = t;
    __syncthreads();
    if (tr == 0 && c < g.N) {
        float s = 0.0f;
        for (int i = 0; i < 16; ++i) s += red[i][tc];
        a.dbias[c] = s;
    }
}

template <typename T>
struct EpiStore {
    T *out;
    int64_t ld;

    template <typename EACH>
    __device__ __forceinline__ void run(EACH each) const {
        each([&](int m, int n, const Vec<float, 8> &v, int cnt) {
            Vec<T, 8> r;
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = from_f32<T>(v.v[e]);
            store_vec_n<T, 8>(out + (int64_t)m * ld + n, r, cnt);
        });
    }
};

template <typename XT, typename YT>
void backward(const LinearGeo &g, const LinearPtrs &p, hipStream_t st) {
    constexpr int V = 16 / (sizeof(XT) > sizeof(YT) ? sizeof(XT) : sizeof(YT));
    if (g.M > 0 && (g.dz_own || p.dbias)) {
        const auto go = [&](auto kernel, int v) {
            const int ncol = (g.N + 64 * v - 1) / (64 * v);
            hipLaunchKernelGGL(kernel, dim3((unsigned)((int64_t)ncol * g.dz_nchunk)), dim3(256), 0, st, g, p, ncol,
                               p.dbias != nullptr);
        };
        if (g.N >= V) go(k_dz<XT, YT, V>, V);
        else go(k_dz<XT, YT, 1>, 1);
    }
    if (p.dbias) hipLaunchKernelGGL(k_dbias, dim3((g.N + 15) / 16), dim3(256), 0, st, g, p);
    const void *dz = g.dz_own ? p.dz : p.dy;
    const int64_t ldz = g.dz_own ? g.N : g.ys;
    GemmArgs a = {};
    if (p.dx) {
        a.A = dz;
        a.lda = ldz;
        a.B = p.w;
        a.ldb = g.K;
        a.M = g.M;
        a.N = g.K;
        a.K = g.N;
        run_gemm<XT, true, false>(g.dx, a, EpiStore<XT>{(XT *)p.dx, g.xs}, p.partial, st);
    }
    if (p.dw) {
        a.A = dz;
        a.lda = ldz;
        a.B = p.x;
        a.ldb = g.xs;
        a.M = g.N;
        a.N = g.K;
        a.K = g.M;
        run_gemm<XT, false, false>(g.dw, a, EpiStore<XT>{(XT *)p.dw, g.K}, p.partial, st);
    }
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
