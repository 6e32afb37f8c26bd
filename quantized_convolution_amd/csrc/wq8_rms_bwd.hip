// Backward of the root-mean-square norm.
//   n = h rstd;  t = gamma dy;  dx = rstd (t - n mean(t n)) + dh;  dgamma = sum_r dy n
// A block goes through its rows a wave (or a block) each, held in registers:
// one read of dy, h and dh, one write of dx. A thread has the same columns of
// every row, so dgamma is summed in its registers, then over the block's waves
// in LDS and over the blocks by a second kernel, in a fixed order.
// Memory bounds it: with the parts of dgamma 8192 x 1280 bf16 takes 21 us (84 MB,
// 4.0 TB/s), 32768 x 1280 70 (4.8), 8192 x 16000 221 (4.8), 1001 x 333 f32 7.6, of
// which two launches are 5.4. A row of 9000 read twice instead: 222 us for 145.
#include "wq8_rows.h"

namespace wq8 {
namespace {

// The same values, of which the compiler knows nothing.
template <typename T>
__device__ __forceinline__ void forget(Vec<T, kV> &v) {
    uint32_t w[sizeof v / 4];
    __builtin_memcpy(w, &v, sizeof v);
#pragma unroll
    for (int i = 0; i < (int)(sizeof v / 4); ++i) asm("" : "+v"(w[i]));
    __builtin_memcpy(&v, w, sizeof v);
}

// What a thread adds to sum t n: 8 columns.
template <typename XT, typename YT>
__device__ __forceinline__ float dot(const Vec<XT, kV> &h, const Vec<YT, kV> &dy, const Vec<float, kV> &gm, float rstd) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kV; ++k) sum = fmaf(gm.v[k] * to_f32(dy.v[k]), to_f32(h.v[k]) * rstd, sum);
    return sum;
}

template <typename XT, typename YT>
__device__ __forceinline__ Vec<XT, kV> grad(const Vec<XT, kV> &h, const Vec<YT, kV> &dy, const Vec<float, kV> &gm,
                                            const Vec<XT, kV> &dh, bool more, float rstd, float mean) {
    Vec<XT, kV> o;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
        float v = rstd * fmaf(-(to_f32(h.v[k]) * rstd), mean, gm.v[k] * to_f32(dy.v[k]));
        if (more) v += to_f32(dh.v[k]);
        o.v[k] = from_f32<XT>(v);
    }
    return o;
}

template <typename XT, typename YT, int L, int U>
__global__ __launch_bounds__(L < 256 ? 256 : L, L == 64 && U == 3 ? 3 : 1) void k_rms_bwd(RowsGeo g, RmsPtrs a, int want_dgamma) {
    constexpr int PER = L < 256 ? 256 / L : 1;
    __shared__ float red[L > 64 ? 4 * L / 64 : 1];
    __shared__ float join[PER > 1 ? (PER - 1) * U * L * kV : 1];
    const int t = threadIdx.x % L, w = threadIdx.x / L;
    Vec<float, kV> gm[U];
    float dg[U][kV] = {};
    load_gamma<L, U>(gm, a.gamma, t, g.C);
    const int r0 = blockIdx.x * g.chunk, r1 = r0 + min(g.chunk, g.rows - r0);  // r0 + chunk may pass 2^31
    int turn = 0;
    for (int i = r0 + (L < 256 ? w : 0); i < r1; i += PER) {
        Vec<XT, kV> h[U], dh[U];
        Vec<YT, kV> dy[U];
        load_row<XT, L, U>(h, (const XT *)a.x + i * g.xs, t, g.C);
        load_row<YT, L, U>(dy, (const YT *)a.dy + i * g.ys, t, g.C);
        if (a.dh) load_row<XT, L, U>(dh, (const XT *)a.dh + i * g.xs, t, g.C);
        const float rstd = a.rstd_in[i];
        float sum = 0.0f;
        uint32_t none = 0;
#pragma unroll
        for (int s = 0; s < U; ++s) sum += dot(h[s], dy[s], gm[s], rstd);
        reduce_row<L>(sum, none, red, turn++);
        const float mean = sum / (float)g.C;
        // what comes next is formed from the values again: held over the sum it
        // would take the registers of another wave
#pragma unroll
        for (int s = 0; s < U; ++s) {
            forget(h[s]);
            forget(dy[s]);
        }
#pragma unroll
        for (int s = 0; s < U; ++s) {
            store_step<XT, L, U>((XT *)a.dx + i * g.xs, s, t, g.C, grad(h[s], dy[s], gm[s], dh[s], a.dh != nullptr, rstd, mean));
#pragma unroll
            for (int k = 0; k < kV; ++k) dg[s][k] = fmaf(to_f32(dy[s].v[k]), to_f32(h[s].v[k]) * rstd, dg[s][k]);
        }
    }
    if (!want_dgamma) return;
    if constexpr (PER > 1) {
        if (w > 0)
#pragma unroll
            for (int s = 0; s < U; ++s)
#pragma unroll
                for (int k = 0; k < kV; ++k) join[(((w - 1) * U + s) * kV + k) * L + t] = dg[s][k];
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int k = 0; k < kV; ++k)
#pragma unroll
                for (int v = 0; v < PER - 1; ++v) dg[s][k] += join[((v * U + s) * kV + k) * L + t];
    }
#pragma unroll
    for (int s = 0; s < U; ++s) {
        const int c = (s * L + t) * kV;
        Vec<float, kV> o;
#pragma unroll
        for (int k = 0; k < kV; ++k) o.v[k] = dg[s][k];
        if (c < g.C) store_cols<float>(a.part + (int64_t)blockIdx.x * g.C, c, g.C, o);
    }
}

// Rows that no block holds, and those of fewer columns than a vector: dx in two
// passes over each, and dgamma's parts in a
// third, a block for 2048 columns of its rows.
template <typename XT, typename YT>
__global__ __launch_bounds__(1024) void k_rms_bwd_long(RowsGeo g, RmsPtrs a, int blocks) {
    constexpr int L = 1024;
    __shared__ float red[2 * L / 64];
    int b;
    if (!block_number(blocks, b)) return;
    const XT *const h = (const XT *)a.x + (int64_t)b * g.xs, *const dh = (const XT *)a.dh + (int64_t)b * g.xs;
    const YT *const dy = (const YT *)a.dy + (int64_t)b * g.ys;
    const auto gamma = [&](int c) {
        Vec<float, kV> r;
        if (a.gamma) return load_any<float>(a.gamma, c, g.C);
#pragma unroll
        for (int k = 0; k < kV; ++k) r.v[k] = 1.0f;
        return r;
    };
    const float rstd = a.rstd_in[b];
    float sum = 0.0f;
    uint32_t none = 0;
    for (int c = threadIdx.x * kV; c < g.C; c += L * kV)
        sum += dot(load_any<XT>(h, c, g.C), load_any<YT>(dy, c, g.C), gamma(c), rstd);
    reduce_row<L>(sum, none, red, 0);
    const float mean = sum / (float)g.C;
    for (int c = threadIdx.x * kV; c < g.C; c += L * kV) {
        Vec<XT, kV> more = {};
        if (a.dh) more = load_any<XT>(dh, c, g.C);
        store_cols<XT>((XT *)a.dx + (int64_t)b * g.xs, c, g.C,
                       grad(load_any<XT>(h, c, g.C), load_any<YT>(dy, c, g.C), gamma(c), more, a.dh != nullptr, rstd, mean));
    }
}

template <typename XT, typename YT>
__global__ __launch_bounds__(256) void k_rms_dgamma_long(RowsGeo g, RmsPtrs a) {
    const int c = (blockIdx.y * 256 + threadIdx.x) * kV;
    if (c >= g.C) return;
    const int r0 = blockIdx.x * g.chunk, r1 = r0 + min(g.chunk, g.rows - r0);
    Vec<float, kV> o = {};
    for (int i = r0; i < r1; ++i) {
        const Vec<XT, kV> h = load_any<XT>((const XT *)a.x + i * g.xs, c, g.C);
        const Vec<YT, kV> dy = load_any<YT>((const YT *)a.dy + i * g.ys, c, g.C);
        const float rstd = a.rstd_in[i];
#pragma unroll
        for (int k = 0; k < kV; ++k) o.v[k] = fmaf(to_f32(dy.v[k]), to_f32(h.v[k]) * rstd, o.v[k]);
    }
    store_cols<float>(a.part + (int64_t)blockIdx.x * g.C, c, g.C, o);
}

// dgamma from the blocks' parts: 16 columns a block, 64 threads along the parts.
__global__ __launch_bounds__(1024) void k_rms_dgamma(RowsGeo g, RmsPtrs a) {
    __shared__ float red[64][17];
    const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4, c = blockIdx.x * 16 + tc;
    float t = 0.0f;
    if (c < g.C)
#pragma unroll 8
        for (int i = tr; i < g.nchunk; i += 64) t += a.part[(int64_t)i * g.C + c];
    red[tr][tc] = t;
    __syncthreads();
    if (tr < 8) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[tr * 8 + i][tc];
        red[tr * 8][tc] = s;
    }
    __syncthreads();
    if (tr == 0 && c < g.C) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += red[i * 8][tc];
        a.dgamma[c] = s;
    }
}

template <typename XT, typename YT>
void backward(const RowsGeo &g, const RmsPtrs &p, hipStream_t st) {
    if (g.rows > 0) {
        const auto go = [&](auto kernel, int threads) {
            hipLaunchKernelGGL(kernel, dim3(g.nchunk), dim3(threads), 0, st, g, p, p.dgamma != nullptr);
        };
        if (g.s.lanes == 64) {
            if (g.s.unroll == 1) go(k_rms_bwd<XT, YT, 64, 1>, 256);
            else if (g.s.unroll == 2) go(k_rms_bwd<XT, YT, 64, 2>, 256);
            else if (g.s.unroll == 3) go(k_rms_bwd<XT, YT, 64, 3>, 256);
            else go(k_rms_bwd<XT, YT, 64, 4>, 256);
        } else if (g.s.lanes == 256) {
            go(k_rms_bwd<XT, YT, 256, 2>, 256);
        } else if (g.s.lanes == 512) {
            go(k_rms_bwd<XT, YT, 512, 2>, 512);
        } else if (g.s.lanes == 1024) {
            go(k_rms_bwd<XT, YT, 1024, 2>, 1024);
        } else {
            hipLaunchKernelGGL((k_rms_bwd_long<XT, YT>), grid_of(g.rows), dim3(1024), 0, st, g, p, g.rows);
            if (p.dgamma)
                hipLaunchKernelGGL((k_rms_dgamma_long<XT, YT>), dim3(g.nchunk, (g.C + 256 * kV - 1) / (256 * kV)), dim3(256), 0,
                                   st, g, p);
        }
    }
    if (p.dgamma) hipLaunchKernelGGL(k_rms_dgamma, dim3((g.C + 15) / 16), dim3(1024), 0, st, g, p);
}

}  // namespace

wq8_status launch_rms_backward(const RowsGeo &g, wq8_dtype xdt, wq8_dtype ydt, const RmsPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (xdt == WQ8_F32) {
        if (ydt == WQ8_F32) backward<float, float>(g, p, st);
        else backward<float, bf16_t>(g, p, st);
    } else {
        if (ydt == WQ8_F32) backward<bf16_t, float>(g, p, st);
        else backward<bf16_t, bf16_t>(g, p, st);
    }
    return check_launch("root-mean-square norm backward");
}

}  // namespace wq8
