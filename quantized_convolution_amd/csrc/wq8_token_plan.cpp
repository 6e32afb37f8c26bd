// Plans and entry points of the operators on 8-bit codes: argument checks,
// launch shapes and workspace layouts. Nothing is enqueued when a check fails.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <initializer_list>
#include <new>

#include "wq8_token_internal.h"

using namespace wq8;

namespace {

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
    if (have < want) return fail(WQ8_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", have, want);
    return need(ws, "workspace");
}

// Whether `out` is one of the buffers of a call: they must not overlap.
wq8_status apart(const void *out, const char *name, std::initializer_list<const void *> others) {
    if (out)
        for (const void *o : others)
            if (o == out) return fail(WQ8_ERR_INVALID_ARG, "%s must not overlap another buffer", name);
    return WQ8_OK;
}

bool is_dtype(int t) { return t == WQ8_F32 || t == WQ8_BF16; }
bool is_act(int a) { return a >= WQ8_ACT_NONE && a <= WQ8_ACT_GELU_TANH; }

constexpr int64_t kMaxColumns = (int64_t)1 << 20;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;
// A product's backward has lines of its rows' codes, 256 of which are addressed in 32 bits.
constexpr int64_t kMaxProductRows = (int64_t)1 << 24;

wq8_status check_rows(int64_t rows, int C, int x_stride, int y_stride, int64_t most) {
    if (rows < 0 || C < 1) return fail(WQ8_ERR_INVALID_ARG, "sizes must be positive (rows=%lld, columns %d)", (long long)rows, C);
    if ((x_stride && x_stride < C) || (y_stride && y_stride < C))
        return fail(WQ8_ERR_INVALID_ARG, "a row stride is shorter than a row of %d", C);
    if (rows >= most || C >= kMaxColumns) return fail(WQ8_ERR_UNSUPPORTED, "%lld rows, or 2^20 columns, or more", (long long)most);
    return WQ8_OK;
}

// How a row of C columns is held: by as few threads as hold it in registers.
RowShape forward_shape(int C) {
    const int stride = code_stride(C);
    if (C < 8) return {0, 0, 1};
    for (int steps : {1, 2, 3, 4, 5, 6, 8})
        if (stride <= 512 * steps) return {64, steps, 4};
    for (int steps : {3, 4, 5, 8})
        if (stride <= 2048 * steps) return {256, steps, 1};
    if (stride <= 32768) return {1024, 4, 1};
    return {0, 0, 1};
}

RowShape backward_shape(int C) {
    const int stride = code_stride(C);
    if (C < 8) return {0, 0, 1};
    for (int steps : {1, 2, 3, 4})
        if (stride <= 512 * steps) return {64, steps, 4};
    if (stride <= 4096) return {256, 2, 1};
    if (stride <= 8192) return {512, 2, 1};
    if (stride <= 16384) return {1024, 2, 1};
    return {0, 0, 1};
}

void set_rows(RowsGeo &g, int64_t rows, int C, int64_t xs, int64_t ys) {
    g.rows = (int)rows;
    g.C = C;
    g.stride = code_stride(C);
    g.xs = xs ? xs : C;
    g.ys = ys ? ys : C;
}

wq8_status build_quant(const wq8_quant_desc *d, wq8_quant_plan *p) {
    WQ8_TRY(check_rows(d->rows, d->C, d->x_stride, 0, kMaxRows));
    if (d->group != 0 && d->group != 32 && d->group != 64 && d->group != 128)
        return fail(WQ8_ERR_INVALID_ARG, "group is 0, 32, 64 or 128, not %d", d->group);
    if (!is_dtype(d->x_dtype)) return fail(WQ8_ERR_INVALID_ARG, "unknown dtype");
    RowsGeo &g = p->geo;
    set_rows(g, d->rows, d->C, d->x_stride, 0);
    g.group = d->group;
    g.s = forward_shape(g.C);
    p->xdt = d->x_dtype;
    if (ceil_div((int64_t)g.rows * (g.stride / 8), 256) >= (int64_t)1 << 31)
        return fail(WQ8_ERR_UNSUPPORTED, "more than 2^31 blocks");
    return WQ8_OK;
}

wq8_status build_rms(const wq8_rms_desc *d, wq8_rms_plan *p) {
    WQ8_TRY(check_rows(d->rows, d->C, d->x_stride, d->y_stride, kMaxRows));
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return fail(WQ8_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (!is_dtype(d->x_dtype) || !is_dtype(d->y_dtype)) return fail(WQ8_ERR_INVALID_ARG, "unknown dtype");
    set_rows(p->f, d->rows, d->C, d->x_stride, d->y_stride);
    p->f.eps = d->eps;
    p->b = p->f;
    p->f.s = forward_shape(p->f.C);
    RowsGeo &g = p->b;
    g.s = backward_shape(g.C);
    // as many blocks as run at once by their registers (8192 x 5120 bf16, two a compute
    // unit: 78 us, with three 97, with one 103), but no more than 256 of fewer than four
    // rows: each has a part of dgamma to be joined (1001 x 2560 bf16 12.8 us, with one
    // row a block 18.1)
    const int L = g.s.lanes, U = g.s.unroll, units = L == 0 || L == 1024 ? 1 : L == 512 || U == 4 ? 2 : U == 3 ? 3 : 4;
    g.chunk = (int)round_up(ceil_div(g.rows, units * kCus), g.s.per);
    const int least = (int)ceil_div(g.rows, kCus);
    if (g.chunk < 4) g.chunk = least < 4 ? (g.chunk < least ? least : g.chunk) : 4;
    g.nchunk = g.rows ? (int)ceil_div(g.rows, g.chunk) : 0;
    p->xdt = d->x_dtype;
    p->ydt = d->y_dtype;
    p->b_bytes = (size_t)g.nchunk * g.C * 4;
    return WQ8_OK;
}

// ------------------------------------------------------ product's launch shape
// Tiles and splits by the least modelled time, as the bf16 product's plan has it,
// at the rates of the int8 matrix cores.
struct Product {
    int64_t M, N, steps;
};

// The forward's kernel for short batches: microseconds of its blocks of 32 rows by
// 32 columns, two a compute unit, whose waves take a quarter of the k steps each.
// A round that leaves units with one block is half as long; a step takes 0.22 us
// where no block has a neighbour, 0.5 where one round has it all, 0.7 in many. What
// it reads through the caches comes at 17 TB/s at best, the weights at 5.5. 64 rows
// of 5120 x 5120 take 7.8 us so and 11.9 in the best tile, 512 rows 38.8 and 26.0.
double thin_us(const Product &q) {
    const double blocks = (double)(ceil_div(q.M, q.M <= 16 ? 16 : 32) * ceil_div(q.N, 32)), steps = (double)ceil_div(q.steps, 4);
    const double halves = ceil(blocks / kCus);
    const double us = halves <= 1 ? 0.22 * steps : halves <= 2 ? 0.5 * steps : halves / 2 * (2.0 + 0.7 * steps) - 2.2;
    const double read = fmax(blocks * 64 / 17.0, (double)q.N / 5.5) * (double)q.steps * 128e-6;
    return 2.2 + fmax(us, read);
}

void choose_q8(const Product *q, int count, int planes, Q8Shape *const *out) {
    constexpr int kMost = 16;
    double least = 1e30;
    const bool pair = planes > 1;
    if (!pair && q[0].steps <= kQ8MaxSteps) {
        least = thin_us(q[0]);
        *out[0] = {kQ8Thin, 1, (int)q[0].steps};
    }
    for (int i = 0; i < 4; ++i) {
        const Q8Tile &g = pair ? kQ8PairTiles[i] : kQ8Tiles[i];
        const double rate = 9.5 * g.rate;  // M operations per us and compute unit
        // a step's loads, barrier and LDS reads take a quarter of a microsecond
        const double step = fmax(2e-6 * g.bm * g.bn * 128 * planes / rate, 0.25 * (planes > 2 ? 2 : 1));
        for (int combo = 0; combo < (count == 1 ? kMost : kMost * kMost); ++combo) {
            const int64_t more[2] = {combo % kMost, combo / kMost};
            int64_t blocks = 0, work = 0, longest = 0, per[2] = {0, 0}, sp[2] = {1, 1};
            double join = 0.0;
            bool fits = true;
            for (int j = 0; j < count; ++j) {
                const int64_t steps = q[j].steps, want = (steps > 0 ? ceil_div(steps, kQ8MaxSteps) : 1) + more[j];
                if (more[j] > 0 && want * 2 > steps) fits = false;
                per[j] = steps ? ceil_div(steps, want) : 0;
                sp[j] = steps ? ceil_div(steps, per[j]) : 1;
                if (sp[j] != want && more[j] > 0) fits = false;
                const int64_t n = ceil_div(q[j].M, g.bm) * ceil_div(q[j].N, g.bn) * sp[j];
                blocks += n;
                work += n * per[j];
                if (per[j] > longest) longest = per[j];
                if (sp[j] > 1) join += (double)q[j].M * q[j].N * 8e-6 * sp[j] / 5.0;
            }
            if (!fits) continue;
            const int64_t n = ceil_div(blocks, kCus);
            double us = count == 1 ? (double)n * longest * step : (double)ceil_div(work, kCus) * step + 0.25 * longest * step;
            if (us < longest * step) us = longest * step;
            if (!pair) us = fmax(us, (double)(q[0].M + q[0].N) * (double)q[0].steps * 128e-6 / 5.5);  // read from memory
            if (n == 1 && g.blocks > 1) us *= 1.3;
            us += (double)ceil_div(n, g.blocks) * (i == 0 ? 10.0 : i == 1 ? 4.0 : 2.5);
            if (join > 0.0) us += (count == 1 ? 3.0 : 5.0) + join;
            if (us < least) {
                least = us;
                for (int j = 0; j < count; ++j) *out[j] = {i, (int)sp[j], (int)per[j]};
            }
        }
    }
}

wq8_status build_q8linear(const wq8_q8linear_desc *d, wq8_q8linear_plan *p) {
    WQ8_TRY(check_rows(d->rows, d->Cin, d->x_stride, 0, kMaxProductRows));
    WQ8_TRY(check_rows(d->rows, d->Cout, d->y_stride, d->r_stride, kMaxProductRows));
    if (!is_act(d->act)) return fail(WQ8_ERR_INVALID_ARG, "unknown activation %d", (int)d->act);
    if (!is_dtype(d->x_dtype) || !is_dtype(d->y_dtype)) return fail(WQ8_ERR_INVALID_ARG, "unknown dtype");
    if (d->r_layout != WQ8_NHWC && d->r_layout != WQ8_NCHW) return fail(WQ8_ERR_INVALID_ARG, "unknown layout");
    if (d->r_layout == WQ8_NCHW && (d->pixels < 1 || d->rows % d->pixels != 0))
        return fail(WQ8_ERR_INVALID_ARG, "rows = %lld is not a multiple of pixels = %d", (long long)d->rows, d->pixels);
    if (d->r_stride && d->r_layout == WQ8_NCHW) return fail(WQ8_ERR_INVALID_ARG, "a row stride is given for an NCHW residual");
    Q8Geo &g = p->geo;
    g.M = (int)d->rows;
    g.K = d->Cin;
    g.N = d->Cout;
    g.Mp = code_stride(g.M);
    g.Kp = code_stride(g.K);
    g.Np = code_stride(g.N);
    g.act = d->act;
    g.xs = d->x_stride ? d->x_stride : d->Cin;
    g.ys = d->y_stride ? d->y_stride : d->Cout;
    g.rs = d->r_stride ? d->r_stride : d->Cout;
    g.r_planar = d->r_layout == WQ8_NCHW;
    g.pixels = d->pixels;
    p->xdt = d->x_dtype;
    p->ydt = d->y_dtype;
    g.planes = p->xdt == WQ8_BF16 && d->round_dz ? 2 : 4;
    const int64_t steps = g.Kp / 128;
    // two rows at most: 3.1 us for 1280 x 1280, 17.6 for 10240 x 10240, where the
    // kernel for short batches takes 3.4 and 18.8; at three rows 3.8 and 18.2, and
    // 7.6 for 5120 x 5120 where that takes 5.0
    if (g.M <= 2 && steps <= kQ8MaxSteps) {
        g.f = {kQ8Rows, 1, (int)steps};
    } else {
        const Product f = {g.M, g.N, steps};
        Q8Shape *const fs[1] = {&g.f};
        choose_q8(&f, 1, 1, fs);
    }
    const Product bwd[2] = {{g.N, g.K, g.Mp / 128}, {g.M, g.K, g.Np / 128}};
    Q8Shape *const bs[2] = {&g.dw, &g.dx};
    choose_q8(bwd, 2, g.planes, bs);
    // rows per block of the first pass: 8 waves of 2 rows in flight, blocks that all
    // run at once, two a compute unit by their registers
    g.ncol = (int)ceil_div(g.N, 512);
    g.chunk = (int)round_up(ceil_div(g.M, 2 * kCus > g.ncol ? 2 * kCus / g.ncol : 1), 16);
    if (g.chunk < 16) g.chunk = 16;
    g.nchunk = (int)ceil_div(g.M, g.chunk);
    const auto tiles = [](const Q8Shape &s, const Q8Tile *t, int64_t M, int64_t N) {
        if (s.tile == kQ8Rows) return ceil_div(N, 8);
        if (s.tile == kQ8Thin) return ceil_div(M, 16) * ceil_div(N, 32);
        return ceil_div(M, t[s.tile].bm) * ceil_div(N, t[s.tile].bn) * s.splits;
    };
    const int64_t lim = (int64_t)1 << 31;
    const int64_t lines = (int64_t)(g.Mp / 128) * (g.Kp / 128) + (int64_t)(g.Np / 128) * (g.Kp / 128);
    if (tiles(g.f, kQ8Tiles, g.M, g.N) >= lim ||
        tiles(g.dx, kQ8PairTiles, g.M, g.K) + tiles(g.dw, kQ8PairTiles, g.N, g.K) + g.N >= lim ||
        (int64_t)g.nchunk * g.ncol + lines >= lim || (int64_t)(g.Mp / 128) * (g.Np / 32) >= lim ||
        ceil_div(g.M, 16) * ceil_div(g.N > g.K ? g.N : g.K, 128) >= lim)
        return fail(WQ8_ERR_UNSUPPORTED, "more than 2^31 blocks");
    const size_t M = g.M, N = g.N, K = g.K;
    const auto partial = [](const Q8Shape &s, size_t m, size_t n) { return s.splits > 1 ? s.splits * m * n * 4 : 0; };
    p->f_bytes = partial(g.f, M, N);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t from = at;
        at += round_up(bytes, 256);
        return from;
    };
    p->off_partial_dx = take(partial(g.dx, M, K));
    p->off_partial_dw = take(partial(g.dw, N, K));
    p->off_xt = take(K * g.Mp);
    p->off_wt = take(K * g.Np);
    p->off_ur = take((size_t)g.planes * M * g.Np);
    p->off_uc = take((size_t)g.planes * N * g.Mp);
    p->off_rowmax = take(M * g.ncol * 4);
    p->off_colmax = take((size_t)g.nchunk * g.Np * 4);
    p->off_colsum = take((size_t)g.nchunk * g.Np * 4);
    p->off_rscale = take(M * 4);
    p->off_cscale = take(N * 4);
    p->b_bytes = g.M ? at : 0;
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

template <typename P>
wq8_status query(const P *p, size_t *forward_bytes, size_t *backward_bytes) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (forward_bytes) *forward_bytes = p->f_bytes;
    if (backward_bytes) *backward_bytes = p->b_bytes;
    return WQ8_OK;
}

}  // namespace

extern "C" {

wq8_status wq8_quant_plan_create(const wq8_quant_desc *desc, wq8_quant_plan **out) { return create(desc, out, build_quant); }

void wq8_quant_plan_destroy(wq8_quant_plan *plan) { delete plan; }

wq8_status wq8_quant_pack(const wq8_quant_plan *p, const void *x, int8_t *codes, float *scales, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.rows == 0) return WQ8_OK;
    WQ8_NEED(x);
    WQ8_NEED(codes);
    WQ8_NEED(scales);
    WQ8_TRY(apart(codes, "codes", {x, scales}));
    WQ8_TRY(apart(scales, "scales", {x}));
    return (p->geo.group ? launch_pack_groups : launch_pack_rows)(p->geo, p->xdt, x, codes, scales, stream);
}

wq8_status wq8_quant_unpack(const wq8_quant_plan *p, const int8_t *codes, const float *scales, void *x, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.rows == 0) return WQ8_OK;
    WQ8_NEED(codes);
    WQ8_NEED(scales);
    WQ8_NEED(x);
    WQ8_TRY(apart(x, "x", {codes, scales}));
    return launch_unpack(p->geo, p->xdt, codes, scales, x, stream);
}

wq8_status wq8_rms_plan_create(const wq8_rms_desc *desc, wq8_rms_plan **out) { return create(desc, out, build_rms); }

void wq8_rms_plan_destroy(wq8_rms_plan *plan) { delete plan; }

wq8_status wq8_rms_plan_query(const wq8_rms_plan *p, size_t *forward_bytes, size_t *backward_bytes) {
    return query(p, forward_bytes, backward_bytes);
}

wq8_status wq8_rms_forward(const wq8_rms_plan *p, const void *x, const void *residual, const float *gamma, void *h, void *y,
                           int8_t *codes, float *scales, float *rstd, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->f.rows == 0) return WQ8_OK;
    if (!y && !codes) return fail(WQ8_ERR_INVALID_ARG, "y or codes must be given");
    if (!codes != !scales) return fail(WQ8_ERR_INVALID_ARG, "codes and scales come together");
    if (h && !residual) return fail(WQ8_ERR_INVALID_ARG, "h is x itself without a residual");
    WQ8_NEED(x);
    WQ8_OPTIONAL(residual);
    WQ8_OPTIONAL(gamma);
    WQ8_OPTIONAL(h);
    WQ8_OPTIONAL(y);
    WQ8_OPTIONAL(codes);
    WQ8_OPTIONAL(scales);
    WQ8_OPTIONAL(rstd);
    WQ8_TRY(apart(y, "y", {x, residual, gamma, h, codes, scales, rstd}));
    WQ8_TRY(apart(h, "h", {gamma, codes, scales, rstd}));
    WQ8_TRY(apart(codes, "codes", {x, residual, gamma, scales, rstd}));
    WQ8_TRY(apart(scales, "scales", {x, residual, gamma, rstd}));
    WQ8_TRY(apart(rstd, "rstd", {x, residual, gamma}));
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->f_bytes));
    RmsPtrs a;
    memset(&a, 0, sizeof a);
    a.x = x;
    a.residual = residual;
    a.gamma = gamma;
    a.h = h;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    a.rstd = rstd;
    return launch_rms_forward(p->f, p->xdt, p->ydt, a, stream);
}

wq8_status wq8_rms_backward(const wq8_rms_plan *p, const void *dy, const void *h, const float *rstd, const float *gamma,
                            const void *dh, void *dx, float *dgamma, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->b.rows > 0) {
        WQ8_NEED(dy);
        WQ8_NEED(h);
        WQ8_NEED(rstd);
        WQ8_OPTIONAL(gamma);
        WQ8_OPTIONAL(dh);
        WQ8_NEED(dx);
        WQ8_TRY(apart(dx, "dx", {dy, h, rstd, gamma, dgamma}));
    }
    WQ8_OPTIONAL(dgamma);
    WQ8_TRY(apart(dgamma, "dgamma", {dy, h, rstd, gamma, dh}));
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->b_bytes));
    RmsPtrs a;
    memset(&a, 0, sizeof a);
    a.dy = dy;
    a.x = h;
    a.rstd_in = rstd;
    a.gamma = gamma;
    a.dh = dh;
    a.dx = dx;
    a.dgamma = dgamma;
    a.part = (float *)workspace;
    return launch_rms_backward(p->b, p->xdt, p->ydt, a, stream);
}

wq8_status wq8_q8linear_plan_create(const wq8_q8linear_desc *desc, wq8_q8linear_plan **out) {
    return create(desc, out, build_q8linear);
}

void wq8_q8linear_plan_destroy(wq8_q8linear_plan *plan) { delete plan; }

wq8_status wq8_q8linear_plan_query(const wq8_q8linear_plan *p, size_t *forward_bytes, size_t *backward_bytes) {
    return query(p, forward_bytes, backward_bytes);
}

wq8_status wq8_q8linear_forward(const wq8_q8linear_plan *p, const int8_t *xq, const float *sx, const int8_t *wq, const float *sw,
                                const float *bias, const void *residual, void *y, void *z, int8_t *zq, float *sz, void *workspace,
                                size_t workspace_bytes, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.M == 0) return WQ8_OK;
    if (!zq != !sz) return fail(WQ8_ERR_INVALID_ARG, "zq and sz come together");
    WQ8_NEED(xq);
    WQ8_NEED(sx);
    WQ8_NEED(wq);
    WQ8_NEED(sw);
    WQ8_OPTIONAL(bias);
    WQ8_OPTIONAL(residual);
    WQ8_NEED(y);
    WQ8_OPTIONAL(z);
    WQ8_OPTIONAL(zq);
    WQ8_OPTIONAL(sz);
    WQ8_TRY(apart(y, "y", {xq, sx, wq, sw, bias, z, zq, sz}));
    WQ8_TRY(apart(z, "z", {xq, sx, wq, sw, bias, residual, zq, sz}));
    WQ8_TRY(apart(zq, "zq", {xq, sx, wq, sw, bias, residual, sz}));
    WQ8_TRY(apart(sz, "sz", {xq, sx, wq, sw, bias, residual}));
    if (y == residual && (p->geo.r_planar || p->geo.rs != p->geo.ys))
        return fail(WQ8_ERR_INVALID_ARG, "a residual that is y itself needs y's layout and row stride");
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->f_bytes));
    Q8Ptrs a;
    memset(&a, 0, sizeof a);
    a.xq = xq;
    a.sx = sx;
    a.wq = wq;
    a.sw = sw;
    a.bias = bias;
    a.residual = residual;
    a.y = y;
    a.z = z;
    a.zq = zq;
    a.sz = sz;
    a.partial = workspace;
    return launch_q8_forward(p->geo, p->ydt, a, stream);
}

wq8_status wq8_q8linear_backward(const wq8_q8linear_plan *p, const void *dy, const int8_t *xq, const float *sx, const int8_t *wq,
                                 const float *sw, const void *z, const int8_t *zq, const float *sz, void *dx, void *dw,
                                 float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    if (!p) return fail(WQ8_ERR_INVALID_ARG, "null plan");
    if (p->geo.M > 0) {
        if (!zq != !sz) return fail(WQ8_ERR_INVALID_ARG, "zq and sz come together");
        WQ8_NEED(dy);
        WQ8_NEED(xq);
        WQ8_NEED(sx);
        WQ8_NEED(wq);
        WQ8_NEED(sw);
        WQ8_OPTIONAL(z);
        WQ8_OPTIONAL(zq);
        WQ8_OPTIONAL(sz);
        if (p->geo.act != WQ8_ACT_NONE && !z == !zq)
            return fail(WQ8_ERR_INVALID_ARG, "z, or zq with sz, must be given: one of the two");
        WQ8_OPTIONAL(dx);
        WQ8_TRY(apart(dx, "dx", {dy, xq, sx, wq, sw, z, zq, sz, dw, dbias}));
    }
    WQ8_OPTIONAL(dw);
    WQ8_OPTIONAL(dbias);
    WQ8_TRY(apart(dw, "dw", {dy, xq, sx, wq, sw, z, zq, sz, dbias}));
    WQ8_TRY(apart(dbias, "dbias", {dy, xq, sx, wq, sw, z, zq, sz}));
    WQ8_TRY(need_workspace(workspace, workspace_bytes, p->b_bytes));
    char *ws = (char *)workspace;
    Q8Ptrs a;
    memset(&a, 0, sizeof a);
    a.dy = dy;
    a.xq = xq;
    a.sx = sx;
    a.wq = wq;
    a.sw = sw;
    a.z_in = z;
    a.zq_in = zq;
    a.sz_in = sz;
    a.dx = dx;
    a.dw = dw;
    a.dbias = dbias;
    a.partial_dx = ws + p->off_partial_dx;
    a.partial_dw = ws + p->off_partial_dw;
    a.xt = (int8_t *)(ws + p->off_xt);
    a.wt = (int8_t *)(ws + p->off_wt);
    a.ur = (int8_t *)(ws + p->off_ur);
    a.uc = (int8_t *)(ws + p->off_uc);
    a.rowmax = (float *)(ws + p->off_rowmax);
    a.colmax = (float *)(ws + p->off_colmax);
    a.colsum = (float *)(ws + p->off_colsum);
    a.rscale = (float *)(ws + p->off_rscale);
    a.cscale = (float *)(ws + p->off_cscale);
    return launch_q8_backward(p->geo, p->xdt, p->ydt, a, stream);
}

}  // extern "C"
