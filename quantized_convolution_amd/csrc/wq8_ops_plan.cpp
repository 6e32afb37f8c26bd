// Plans and entry points of the group norm and the matrix product: argument
// checks, launch shapes and workspace layouts. Nothing is enqueued when a
// check fails.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>

#include "wq8_ops_internal.h"

using namespace wq8;

namespace {

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int ceil_div(int a, int b) { return a / b + (a % b != 0); }
int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

wq8_status need(const void *p, const char *name) {
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)p & 15u) return fail(WQ8_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
    return WQ8_OK;
}

wq8_status optional(const void *p, const char *name) { return p ? need(p, name) : WQ8_OK; }

#define WQ8_TRY(expr)                  \
    do {                               \
        wq8_status _st = (expr);       \
        if (_st != WQ8_OK) return _st; \
    } while (0)
#define WQ8_NEED(p) WQ8_TRY(need((const void *)(p), #p))
#define WQ8_OPTIONAL(p) WQ8_TRY(optional((const void *)(p), #p))

wq8_status need_workspace(const void *ws, size_t have, size_t want) {
    if (want == 0) return WQ8_OK;
    if (have < want)
        return fail(WQ8_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", have, want);
    return need(ws, "workspace");
}

bool is_dtype(int t) { return t == WQ8_F32 || t == WQ8_BF16; }
int size_of(wq8_dtype t) { return t == WQ8_F32 ? 4 : 2; }
bool is_act(int a) { return a >= WQ8_ACT_NONE && a <= WQ8_ACT_GELU_TANH; }
bool is_layout(int l) { return l == WQ8_NHWC || l == WQ8_NCHW; }

// --------------------------------------------------------- norm's launch shape
// The fused shape for slabs of K groups, or steps > most if no block of up to
// 1024 threads holds them.
NormShape fused_shape(const NormGeo &g, int V, int K, int most) {
    NormShape s;
    memset(&s, 0, sizeof s);
    s.V = V;
    s.K = K;
    s.J = 1;
    s.slabC = K * g.cpg;
    s.nslab = g.G / K;
    s.chunk = g.P;
    s.nchunk = 1;
    s.steps = 1 << 30;
    if (s.slabC > kNormMaxSlab) return s;
    // threads across the channels (NHWC) or the channels times the pixel
    // vectors (NCHW); along the rest, as many as take all of the unrolled steps
    // (a block whose steps end with its pixels checks no bounds)
    const int across = g.x_nhwc ? ceil_div(s.slabC, V) : s.slabC;
    const int along = g.x_nhwc ? g.P : ceil_div(g.P, V);
    int lanes = ceil_div(along, kNormE);
    if (across * lanes > 1024) lanes = ceil_div(along, most);
    if (across * lanes > 1024) return s;
    s.steps = ceil_div(along, lanes);
    s.tc = across;
    s.tp = lanes;
    s.window = g.x_nhwc ? lanes : lanes * V;
    s.threads = (int)round_up((size_t)across * lanes, 64);
    return s;
}

// Split shape: blocks of 256 threads that take `batch` steps at a time.
NormShape split_shape(const NormGeo &g, int V, int batch, int xsz) {
    constexpr int T = kNormSplitThreads;
    NormShape s;
    memset(&s, 0, sizeof s);
    s.V = V;
    s.J = 1;
    s.K = 1;
    s.threads = T;
    s.split = 1;
    if (g.x_nhwc) {
        const int across = ceil_div(g.cpg, V), most = kNormMaxSlab / V < T ? kNormMaxSlab / V : T;  // columns
        if (across > most) {
            s.slabC = ceil_div(across, ceil_div(across, most)) * V;
            s.J = ceil_div(g.cpg, s.slabC);
        } else {
            // whole groups: the first count of at least 256 bytes a row that keeps
            // 7 of 8 lanes busy, else the most bytes, else the most lanes (more
            // groups to a block are more parts for it to join)
            double best = -1;
            for (int k = 1; k <= g.G; ++k) {
                const int vecs = ceil_div(k * g.cpg, V);
                if (vecs > most) break;
                if (g.G % k != 0 || k * g.cpg < V) continue;
                const double busy = (double)k * g.cpg / V * (T / vecs) / T;
                if (busy < best && busy < 0.875) continue;
                best = busy;
                s.K = k;
                if (busy >= 0.875 && k * g.cpg * xsz >= 256) break;
            }
            s.slabC = s.K * g.cpg;
        }
        s.tc = ceil_div(s.slabC, V);
        s.tp = T / s.tc;
        if (s.tp > g.P) s.tp = g.P;
        s.window = s.tp;
    } else {
        const int along = ceil_div(g.P, V);
        s.slabC = g.cpg;
        if (g.cpg > T) {
            s.slabC = ceil_div(g.cpg, ceil_div(g.cpg, T));
            s.J = ceil_div(g.cpg, s.slabC);
        }
        s.tc = s.slabC;
        s.tp = T / s.slabC < along ? T / s.slabC : along;
        s.window = s.tp * V;
    }
    s.nslab = g.G / s.K * s.J;
    // one batch of steps to a block, or as many as still leave 8 blocks a
    // compute unit (by their registers 4 to 8 of the statistics' blocks run at
    // once, and 5 or 6 of the output's)
    const int64_t rows = (int64_t)g.N * s.nslab;
    const int all = ceil_div(g.P, s.window);
    int steps = batch;
    while (steps < all && rows * ceil_div(all, steps + batch) >= 8 * kCus) steps += batch;
    if (steps > all) steps = all;
    s.steps = steps;
    const int64_t chunk = (int64_t)s.steps * s.window;
    s.chunk = chunk < g.P ? (int)chunk : g.P;
    s.nchunk = ceil_div(g.P, s.chunk);
    return s;
}

// Whether every position that the kernels form fits 32 bits: a block's last
// batch of steps and its spare threads reach past the image's pixels, and its
// slab past the channels, before they are clamped.
bool positions_fit(const NormGeo &g, const NormShape &s) {
    constexpr int64_t lim = (int64_t)1 << 31, batch = norm_max_steps(false, false, false);
    const int64_t last = (int64_t)(s.nchunk - 1) * s.chunk, most = s.steps + batch;
    return last + s.chunk < lim && last + most * s.window + 1024 * norm_max_vec(2, 2, false) < lim &&
           (int64_t)g.G / s.K * s.J * s.slabC + 2 * kNormMaxSlab < lim;
}

// Steps whose windows fit 48 KiB of LDS (rows padded by two elements), one at
// least: 1024 threads' vectors do.
void set_tile_steps(const NormGeo &g, NormShape &s, int ysz, int batch) {
    const auto bytes = [&](int64_t n) {
        return (g.x_nhwc ? s.slabC * (n * s.window + 2) : n * s.window * (s.slabC + 2)) * ysz;
    };
    s.tsteps = 1;
    while (s.tsteps < batch && s.tsteps < s.steps && bytes(s.tsteps + 1) <= 49152) ++s.tsteps;
}

// Whether some slab of whole groups, or of a group's part, holds a vector of V
// channels and no more than a block may have.
bool slab_holds(const NormGeo &g, int V) {
    for (int k = 1; k <= g.G; ++k)
        if (g.G % k == 0 && k * g.cpg >= V) return k == 1 || k * g.cpg <= kNormMaxSlab;
    return false;
}

NormShape choose_norm(const NormGeo &g, int xsz, int ysz, bool backward) {
    const int vmax = norm_max_vec(xsz, ysz, backward);
    // single values where no row holds a vector
    const bool single = g.x_nhwc ? !slab_holds(g, vmax) : g.P < vmax;
    // vectors within one group where the group's channels allow 8 bytes or more,
    // else vectors that straddle groups
    int V = vmax;
    while (g.x_nhwc && V > 4 && g.cpg % V != 0) V /= 2;
    if (g.x_nhwc && g.cpg % V != 0) V = vmax;
    if (single) V = 1;
    const int most = norm_max_steps(backward, g.x_nhwc && g.cpg % V != 0, g.x_nhwc != g.y_nhwc);
    NormShape s;
    s.steps = 1 << 30;
    for (int k = 1; k <= g.G; ++k) {
        // whole vectors across the slab, nearly
        const int64_t chans = (int64_t)k * g.cpg, vecs = ceil_div64(chans, V) * V;
        if (g.G % k != 0 || (g.x_nhwc && k < g.G && chans * 8 < vecs * 7) || (g.x_nhwc && chans < V)) continue;
        const NormShape t = fused_shape(g, V, k, most);
        if (t.steps > most) break;
        // wider slabs (longer contiguous rows) while the card stays full
        const bool fills = (int64_t)g.N * t.nslab >= kCus && t.slabC * xsz <= 256;
        if (s.steps > most || fills) s = t;
    }
    if (s.steps <= most) {
        // a block holds a group: one pass, if there are blocks enough or little to do
        const int64_t blocks = (int64_t)g.N * s.nslab, values = (int64_t)g.P * s.slabC;
        if (blocks >= kCus / 2 || values <= 16384) {
            set_tile_steps(g, s, ysz, s.steps);
            return s;
        }
    }
    s = split_shape(g, single ? 1 : vmax, kNormE, xsz);
    set_tile_steps(g, s, ysz, kNormE);
    return s;
}

wq8_status build_norm(const wq8_norm_desc *d, wq8_norm_plan *p) {
    if (d->N < 0 || d->C < 1 || d->H < 1 || d->W < 1)
        return fail(WQ8_ERR_INVALID_ARG, "sizes must be positive (N=%d C=%d H=%d W=%d)", d->N, d->C, d->H, d->W);
    if (d->groups < 1 || d->C % d->groups != 0)
        return fail(WQ8_ERR_INVALID_ARG, "C = %d is not a multiple of groups = %d", d->C, d->groups);
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return fail(WQ8_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (!is_act(d->act)) return fail(WQ8_ERR_INVALID_ARG, "unknown activation %d", (int)d->act);
    if (!is_dtype(d->x_dtype) || !is_dtype(d->y_dtype)) return fail(WQ8_ERR_INVALID_ARG, "unknown dtype");
    if (!is_layout(d->x_layout) || !is_layout(d->y_layout)) return fail(WQ8_ERR_INVALID_ARG, "unknown layout");
    const auto stride_ok = [&](int stride, wq8_layout l) { return stride == 0 || (l == WQ8_NHWC && stride >= d->C); };
    if (!stride_ok(d->x_stride, d->x_layout) || !stride_ok(d->y_stride, d->y_layout))
        return fail(WQ8_ERR_INVALID_ARG, "a pixel stride is for NHWC only and at least C = %d (x_stride=%d y_stride=%d)",
                    d->C, d->x_stride, d->y_stride);
    const int64_t lim = (int64_t)1 << 31, P = (int64_t)d->H * d->W;
    // pixels of an image and values of its channels are counted in 32 bits;
    // images and whole tensors are addressed in 64
    if (P * d->C >= lim || (int64_t)d->N * d->groups >= lim || (int64_t)d->N * d->C >= lim)
        return fail(WQ8_ERR_UNSUPPORTED, "an image of 2^31 values or more");
    NormGeo &g = p->geo;
    g.N = d->N;
    g.C = d->C;
    g.P = (int)P;
    g.G = d->groups;
    g.cpg = d->C / d->groups;
    g.eps = d->eps;
    g.act = d->act;
    g.x_nhwc = d->x_layout == WQ8_NHWC;
    g.y_nhwc = d->y_layout == WQ8_NHWC;
    g.xs = d->x_stride ? d->x_stride : d->C;
    g.ys = d->y_stride ? d->y_stride : d->C;
    p->xdt = d->x_dtype;
    p->ydt = d->y_dtype;
    g.f = choose_norm(g, size_of(p->xdt), size_of(p->ydt), false);
    g.b = choose_norm(g, size_of(p->xdt), size_of(p->ydt), true);
    if (!positions_fit(g, g.f) || !positions_fit(g, g.b))
        return fail(WQ8_ERR_UNSUPPORTED, "an image whose last block would pass 2^31 pixels or channels");
    if ((int64_t)g.N * g.f.nslab * g.f.nchunk >= lim || (int64_t)g.N * g.b.nslab * g.b.nchunk >= lim)
        return fail(WQ8_ERR_UNSUPPORTED, "more than 2^31 blocks");
    const size_t N = g.N, G = g.G, C = g.C;
    const size_t fparts = g.f.nchunk * g.f.J, bparts = g.b.nchunk * g.b.J;
    p->f_off_stats = 0;  // mean, rstd where the caller wants none
    p->f_off_part = round_up(N * G * 8, 256);
    p->f_bytes = p->f_off_part + (g.f.split ? N * G * fparts * 8 : 0);
    p->b_off_part = 0;
    p->b_off_group = round_up(N * g.b.nchunk * 3 * C * 4, 256);
    p->b_off_gpart = p->b_off_group + round_up(N * G * 8, 256);
    p->b_bytes = p->b_off_gpart + (g.b.split ? N * G * bparts * 8 : 0);
    return WQ8_OK;
}

// ------------------------------------------------------ product's launch shape
// Tiles and splits by the least modelled time, in microseconds, of one product
// or of two that run side by side in one kernel. A compute unit works through
// its share of the blocks at the tile's rate, a third more slowly where it has
// but one block to itself; each round of blocks that it holds at once adds its
// start and end (much of it for the largest tile, whose compute unit has
// nothing else to do then); a split writes and reads fp32 sums and launches
// once more; with dz in two planes each k step is taken twice. Measured against
// it over 40 shapes and tiles (bf16 8192 x 640 x 640: 13.3, 11.2, 12.7 modelled
// and 13.2, 12.5, 13.4 measured for 128 x 128, 128 x 64, 64 x 64; fp32 2048 x
// 2560 x 1280 in 64 x 64: 120 and 124, split in two 112 and 113).
struct Product {
    int64_t M, N, K;
};

void choose_gemm(const Product *q, int count, wq8_dtype t, int planes, bool direct, GemmShape *const *out) {
    constexpr int kMost = 16;  // splits
    const int64_t kstep = t == WQ8_F32 ? 32 : 64;
    double least = 1e30;
    for (int i = 0; i < count; ++i) memset(out[i], 0, sizeof *out[i]);
    for (int i = direct ? 0 : 1; i < kGemmTileCount; ++i) {
        if (i == 1 && count == 2 && t == WQ8_F32) continue;  // 128 x 64 has the rate in fp32, and finer blocks
        const GemmTile &g = kGemmTiles[i];
        const double rate = t == WQ8_F32 ? 0.56 * g.f32 : 5.2 * g.bf16;  // Mflop per us and compute unit
        const double step = 2e-6 * g.bm * g.bn * kstep * planes / rate;
        for (int combo = 0; combo < (count == 1 ? kMost : kMost * kMost); ++combo) {
            const int64_t want[2] = {combo % kMost + 1, combo / kMost + 1};
            int64_t blocks = 0, work = 0, longest = 0, per[2] = {0, 0}, sp[2] = {1, 1};
            double join = 0.0;
            bool fits = true;
            for (int j = 0; j < count; ++j) {
                const int64_t steps = ceil_div64(q[j].K, kstep);
                if (want[j] > 1 && want[j] * 2 > steps) fits = false;
                per[j] = steps ? ceil_div64(steps, want[j]) : 0;
                sp[j] = steps ? ceil_div64(steps, per[j]) : 1;
                if (sp[j] != want[j]) fits = false;
                const int64_t n = ceil_div64(q[j].M, g.bm) * ceil_div64(q[j].N, g.bn) * sp[j];
                blocks += n;
                work += n * per[j];
                if (per[j] > longest) longest = per[j];
                if (sp[j] > 1) join += (double)q[j].M * q[j].N * 8e-6 * sp[j] / 5.0;
            }
            if (!fits) continue;
            const int64_t n = ceil_div64(blocks, kCus);
            // equal blocks come in whole rounds; of two products' the rest evens out
            double us = count == 1 ? (double)n * longest * step : (double)ceil_div64(work, kCus) * step + 0.5 * longest * step;
            if (us < longest * step) us = longest * step;
            if (n == 1 && g.blocks > 1) us *= 1.3;
            us += (double)ceil_div64(n, g.blocks) * (i == 0 ? 10.0 : i == 1 ? 4.0 : 2.5);
            if (join > 0.0) us += 3.0 + join;
            if (us < least) {
                least = us;
                for (int j = 0; j < count; ++j) {
                    out[j]->tile = i;
                    out[j]->direct = direct;
                    out[j]->splits = (int)sp[j];
                    out[j]->ksteps = (int)per[j];
                }
            }
        }
    }
}

// Whether an operand's k steps can go to LDS directly: rows that start on 16
// bytes, and whole 16-byte units along the rows' index where that is the
// contiguous one (k itself may end anywhere).
bool direct_ok(wq8_dtype t, int64_t ld, bool k_contiguous, int64_t rows) {
    const int64_t unit = t == WQ8_F32 ? 4 : 8;
    return ld % unit == 0 && (k_contiguous || rows % unit == 0);
}

wq8_status build_linear(const wq8_linear_desc *d, wq8_linear_plan *p) {
    if (d->rows < 0 || d->Cin < 1 || d->Cout < 1)
        return fail(WQ8_ERR_INVALID_ARG, "sizes must be positive (rows=%lld Cin=%d Cout=%d)", (long long)d->rows, d->Cin,
                    d->Cout);
    if (!is_act(d->act)) return fail(WQ8_ERR_INVALID_ARG, "unknown activation %d", (int)d->act);
    if (!is_dtype(d->x_dtype) || !is_dtype(d->y_dtype)) return fail(WQ8_ERR_INVALID_ARG, "unknown dtype");
    if (!is_layout(d->r_layout)) return fail(WQ8_ERR_INVALID_ARG, "unknown layout");
    if (d->round_dz != 0 && d->round_dz != 1) return fail(WQ8_ERR_INVALID_ARG, "round_dz is 0 or 1, not %d", d->round_dz);
    if (d->r_layout == WQ8_NCHW && (d->pixels < 1 || d->rows % d->pixels != 0))
        return fail(WQ8_ERR_INVALID_ARG, "rows = %lld is not a multiple of pixels = %d", (long long)d->rows, d->pixels);
    if ((d->x_stride && d->x_stride < d->Cin) || (d->y_stride && d->y_stride < d->Cout) ||
        (d->r_stride && (d->r_layout == WQ8_NCHW || d->r_stride < d->Cout)))
        return fail(WQ8_ERR_INVALID_ARG, "a row stride is shorter than a row, or given for an NCHW residual");
    const int64_t big = (int64_t)1 << 22;
    // rows and tiles are counted in 32 bits, and a tile's rows (256 of 4 bytes
    // a column) are addressed in 32; tensors in 64
    if (d->rows >= ((int64_t)1 << 31) - 1024 || d->Cin >= big || d->Cout >= big || d->x_stride >= big || d->y_stride >= big ||
        d->r_stride >= big)
        return fail(WQ8_ERR_UNSUPPORTED, "2^31 rows, or 2^22 columns, or more");
    LinearGeo &g = p->geo;
    g.M = (int)d->rows;
    g.K = d->Cin;
    g.N = d->Cout;
    g.act = d->act;
    g.xs = d->x_stride ? d->x_stride : d->Cin;
    g.ys = d->y_stride ? d->y_stride : d->Cout;
    g.rs = d->r_stride ? d->r_stride : d->Cout;
    g.r_planar = d->r_layout == WQ8_NCHW;
    g.pixels = d->pixels;
    p->xdt = d->x_dtype;
    p->ydt = d->y_dtype;
    // dy serves as dz where the activation leaves it as it is and the products
    // can read its type
    g.dz_own = g.act != WQ8_ACT_NONE || p->xdt != p->ydt;
    g.dz_planes = p->xdt == WQ8_BF16 && g.dz_own && !d->round_dz ? 2 : 1;
    // rows per block: 4 waves of 4 rows in flight, more where blocks abound
    g.dz_chunk = 64;
    while (g.dz_chunk > 16 && ceil_div64(g.M, g.dz_chunk) * ceil_div64(g.N, 512) < 4 * kCus) g.dz_chunk /= 2;
    g.dz_nchunk = ceil_div(g.M, g.dz_chunk);
    const int64_t ldz = g.dz_own ? g.N : g.ys;
    const wq8_dtype t = p->xdt;
    const Product f = {g.M, g.N, g.K}, bwd[2] = {{g.N, g.K, g.M}, {g.M, g.K, g.N}};  // k of one plane
    GemmShape *const fs[1] = {&g.f}, *const bs[2] = {&g.dw, &g.dx};
    choose_gemm(&f, 1, t, 1, direct_ok(t, g.xs, true, g.M) && direct_ok(t, g.K, true, g.N), fs);
    choose_gemm(bwd, 2, t, g.dz_planes,
                direct_ok(t, ldz, true, g.M) && direct_ok(t, g.K, false, g.K) && direct_ok(t, ldz, false, g.N) &&
                    direct_ok(t, g.xs, false, g.K),
                bs);
    const auto tiles = [](const GemmShape &s, int64_t M, int64_t N) {
        return ceil_div64(M, kGemmTiles[s.tile].bm) * ceil_div64(N, kGemmTiles[s.tile].bn) * s.splits;
    };
    const int64_t lim = (int64_t)1 << 31;
    if (ceil_div64(g.N, 64) * g.dz_nchunk >= lim || tiles(g.f, g.M, g.N) >= lim ||
        tiles(g.dx, g.M, g.K) + tiles(g.dw, g.N, g.K) + g.N >= lim)
        return fail(WQ8_ERR_UNSUPPORTED, "more than 2^31 blocks");
    const size_t M = g.M, N = g.N, K = g.K;
    const auto partial = [](const GemmShape &s, size_t m, size_t n) { return s.splits > 1 ? s.splits * m * n * 4 : 0; };
    p->f_off_partial = 0;
    p->f_bytes = partial(g.f, M, N);
    p->b_off_dz = 0;
    p->b_off_colsum = g.dz_own ? round_up(M * N * size_of(p->xdt) * g.dz_planes, 256) : 0;
    p->b_off_partial = p->b_off_colsum + round_up((size_t)g.dz_nchunk * N * 4, 256);
    p->b_off_partial_dw = p->b_off_partial + round_up(partial(g.dx, M, K), 256);
    p->b_bytes = p->b_off_partial_dw + partial(g.dw, N, K);
    return WQ8_OK;
}

// Makes a plan of type P by f(desc, plan).
template <typename P, typename D>
wq8_status create(const D *desc, P **out, wq8_status (*f)(const D *, P *)) {
    clear_error();
    if (!out) return fail(WQ8_ERR_INVALID_ARG, "null output pointer");
    *out = nullptr;
    if (!desc) return fail(WQ8_ERR_INVALID_ARG, "null descriptor");
    P *p = new (std::nothrow) P;
    if (!p) return fail(WQ8_ERR_NO_MEMORY, "out of host memory");
    memset((void *)p, 0, sizeof *p);
    const wq8_status st = f(desc, p);
    if (st != WQ8_OK) {
        delete p;
        return st;
    }
    *out = p;
    return WQ8_OK;
}

}  // namespace

extern "C" {

wq8_status wq8_norm_plan_create(const wq8_norm_desc *desc, wq8_norm_plan **out) {
    return create(desc, out, build_norm);
}

void wq8_norm_plan_destroy(wq8_norm_plan *plan) { delete plan; }

wq8_status wq8_norm_plan_query(const wq8_norm_plan *p, size_t *forward_bytes, size_t *backward_bytes) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (forward_bytes) *forward_bytes = p->f_bytes;
    if (backward_bytes) *backward_bytes = p->b_bytes;
    return WQ8_OK;
}

wq8_status wq8_norm_forward(const wq8_norm_plan *p, const void *x, const float *shift, const float *gamma,
                            const float *beta, void *y, float *mean, float *rstd, void *workspace,
                            size_t workspace_bytes, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.N == 0) return WQ8_OK;
    WQ8_NEED(x);
    WQ8_OPTIONAL(shift);
    WQ8_OPTIONAL(gamma);
    WQ8_OPTIONAL(beta);
    WQ8_NEED(y);
    WQ8_OPTIONAL(mean);
    WQ8_OPTIONAL(rstd);
    if (x == y) return fail(WQ8_ERR_INVALID_ARG, "x and y must not overlap");
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->f_bytes));
    NormPtrs a;
    memset(&a, 0, sizeof a);
    float *stats = (float *)((char *)workspace + p->f_off_stats);
    a.x = x;
    a.shift = shift;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean ? mean : stats;
    a.rstd = rstd ? rstd : stats + (size_t)p->geo.N * p->geo.G;
    a.part = (float *)((char *)workspace + p->f_off_part);
    if (p->xdt == WQ8_F32)
        return (p->ydt == WQ8_F32 ? launch_norm_forward_f32_f32 : launch_norm_forward_f32_bf16)(p->geo, a, stream);
    return (p->ydt == WQ8_F32 ? launch_norm_forward_bf16_f32 : launch_norm_forward_bf16_bf16)(p->geo, a, stream);
}

wq8_status wq8_norm_backward(const wq8_norm_plan *p, const void *dy, const void *x, const float *shift,
                             const float *gamma, const float *beta, const float *mean, const float *rstd, void *dx,
                             float *dgamma, float *dbeta, float *dshift, void *workspace, size_t workspace_bytes,
                             void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.N > 0) {
        WQ8_NEED(dy);
        WQ8_NEED(x);
        WQ8_OPTIONAL(shift);
        WQ8_OPTIONAL(gamma);
        WQ8_OPTIONAL(beta);
        WQ8_NEED(mean);
        WQ8_NEED(rstd);
        WQ8_NEED(dx);
        WQ8_OPTIONAL(dshift);
        if (dx == x || dx == dy) return fail(WQ8_ERR_INVALID_ARG, "dx must not overlap x or dy");
    }
    WQ8_OPTIONAL(dgamma);
    WQ8_OPTIONAL(dbeta);
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->b_bytes));
    char *ws = (char *)workspace;
    NormPtrs a;
    memset(&a, 0, sizeof a);
    a.dy = dy;
    a.x = x;
    a.shift = shift;
    a.gamma = gamma;
    a.beta = beta;
    a.mean_in = mean;
    a.rstd_in = rstd;
    a.dx = dx;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.dshift = dshift;
    a.part = (float *)(ws + p->b_off_part);
    a.group = (float *)(ws + p->b_off_group);
    a.gpart = (float *)(ws + p->b_off_gpart);
    return (p->xdt == WQ8_F32 ? launch_norm_backward_f32 : launch_norm_backward_bf16)(p->geo, p->ydt, a, stream);
}

wq8_status wq8_linear_plan_create(const wq8_linear_desc *desc, wq8_linear_plan **out) {
    return create(desc, out, build_linear);
}

void wq8_linear_plan_destroy(wq8_linear_plan *plan) { delete plan; }

wq8_status wq8_linear_plan_query(const wq8_linear_plan *p, size_t *forward_bytes, size_t *backward_bytes) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (forward_bytes) *forward_bytes = p->f_bytes;
    if (backward_bytes) *backward_bytes = p->b_bytes;
    return WQ8_OK;
}

wq8_status wq8_linear_forward(const wq8_linear_plan *p, const void *x, const void *w, const float *bias,
                              const void *residual, void *y, void *z, void *workspace, size_t workspace_bytes,
                              void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.M == 0) return WQ8_OK;
    WQ8_NEED(x);
    WQ8_NEED(w);
    WQ8_OPTIONAL(bias);
    WQ8_OPTIONAL(residual);
    WQ8_NEED(y);
    WQ8_OPTIONAL(z);
    if (y == x || y == w || z == y || (z && (z == x || z == w || z == residual)) || (p->geo.r_planar && y == residual))
        return fail(WQ8_ERR_INVALID_ARG, "y and z must not overlap each other or an input");
    if (y == residual && p->geo.rs != p->geo.ys)
        return fail(WQ8_ERR_INVALID_ARG, "a residual that is y itself needs y's row stride");
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->f_bytes));
    LinearPtrs a;
    memset(&a, 0, sizeof a);
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.z = z;
    a.partial = (float *)((char *)workspace + p->f_off_partial);
    return (p->xdt == WQ8_F32 ? launch_linear_forward_f32 : launch_linear_forward_bf16)(p->geo, p->ydt, a, stream);
}

wq8_status wq8_linear_backward(const wq8_linear_plan *p, const void *dy, const void *x, const void *w, const void *z,
                               void *dx, void *dw, float *dbias, void *workspace, size_t workspace_bytes,
                               void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.M > 0) {
        WQ8_NEED(dy);
        if (dw) WQ8_NEED(x);
        if (dx) WQ8_NEED(w);
        if (p->geo.act != WQ8_ACT_NONE) WQ8_NEED(z);
        WQ8_OPTIONAL(dx);
        if (dx && (dx == dy || dx == x || dx == w || dx == z || dx == dw))
            return fail(WQ8_ERR_INVALID_ARG, "dx must not overlap an input or dw");
        if (dw && (dw == dy || dw == x || dw == w || dw == z))
            return fail(WQ8_ERR_INVALID_ARG, "dw must not overlap an input");
    }
    WQ8_OPTIONAL(dw);
    WQ8_OPTIONAL(dbias);
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->b_bytes));
    char *ws = (char *)workspace;
    LinearPtrs a;
    memset(&a, 0, sizeof a);
    a.dy = dy;
    a.x = x;
    a.w = w;
    a.zin = z;
    a.dx = dx;
    a.dw = dw;
    a.dbias = dbias;
    a.dz = p->geo.dz_own ? (void *)(ws + p->b_off_dz) : nullptr;
    a.colsum = (float *)(ws + p->b_off_colsum);
    a.partial_dx = (float *)(ws + p->b_off_partial);
    a.partial_dw = (float *)(ws + p->b_off_partial_dw);
    return launch_linear_backward(p->geo, p->xdt, p->ydt, a, stream);
}

}  // extern "C"
