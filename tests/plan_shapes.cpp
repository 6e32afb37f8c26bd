// Prints the launch shapes that plans choose, one line for each line read:
//   norm N C H W groups x_dtype y_dtype x_layout y_layout
//   linear rows Cin Cout act x_dtype y_dtype x_stride y_stride round_dz
// Built by the host tests from the plan's own source; launches are left out.
#include <stdio.h>

#include "../quantized_convolution_amd/csrc/wq8_ops_plan.cpp"

namespace wq8 {
wq8_status fail(wq8_status st, const char *, ...) { return st; }
void clear_error() {}
#define NORM_FORWARD(name) \
    wq8_status name(const NormGeo &, const NormPtrs &, void *) { return WQ8_OK; }
NORM_FORWARD(launch_norm_forward_f32_f32)
NORM_FORWARD(launch_norm_forward_f32_bf16)
NORM_FORWARD(launch_norm_forward_bf16_f32)
NORM_FORWARD(launch_norm_forward_bf16_bf16)
#define WITH_DTYPE(name, Geo, Ptrs) \
    wq8_status name(const Geo &, wq8_dtype, const Ptrs &, void *) { return WQ8_OK; }
WITH_DTYPE(launch_norm_backward_f32, NormGeo, NormPtrs)
WITH_DTYPE(launch_norm_backward_bf16, NormGeo, NormPtrs)
WITH_DTYPE(launch_linear_forward_f32, LinearGeo, LinearPtrs)
WITH_DTYPE(launch_linear_forward_bf16, LinearGeo, LinearPtrs)
wq8_status launch_linear_backward(const LinearGeo &, wq8_dtype, wq8_dtype, const LinearPtrs &, void *) { return WQ8_OK; }
}  // namespace wq8

// KIND of a norm's kernels: P NCHW, U channels of one group, S straddling groups.
static void print_norm(const char *name, const NormGeo &g, const NormShape &s, bool backward) {
    const char kind = !g.x_nhwc ? 'P' : g.cpg % s.V == 0 ? 'U' : 'S';
    const int unrolled = s.split || s.steps <= kNormE ? kNormE : norm_max_steps(backward, kind == 'S', g.x_nhwc != g.y_nhwc);
    printf("%s=%s%c%d/%d%s batches=%d J=%d ", name, s.split ? "split" : "fused", kind, s.V, unrolled,
           g.x_nhwc != g.y_nhwc ? "x" : "", (s.steps + unrolled - 1) / unrolled, s.J);
}

int main() {
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        int a[10];
        long long rows;
        if (sscanf(line, "norm %d %d %d %d %d %d %d %d %d", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7, a + 8) == 9) {
            const wq8_norm_desc d = {a[0], a[1], a[2], a[3], a[4], 1e-5f, WQ8_ACT_SILU, (wq8_dtype)a[5], (wq8_dtype)a[6],
                                     (wq8_layout)a[7], (wq8_layout)a[8], 0, 0};
            wq8_norm_plan *p;
            if (wq8_norm_plan_create(&d, &p) != WQ8_OK) return 1;
            print_norm("f", p->geo, p->geo.f, false);
            print_norm("b", p->geo, p->geo.b, true);
            printf("\n");
            wq8_norm_plan_destroy(p);
        } else if (sscanf(line, "linear %lld %d %d %d %d %d %d %d %d", &rows, a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7) == 9) {
            const wq8_linear_desc d = {rows, a[0], a[1], (wq8_act)a[2], (wq8_dtype)a[3], (wq8_dtype)a[4], WQ8_NHWC, 0,
                                       a[5], a[6], 0, a[7]};
            wq8_linear_plan *p;
            if (wq8_linear_plan_create(&d, &p) != WQ8_OK) return 1;
            const auto print = [](const char *name, const GemmShape &s) {
                printf("%s=%dx%d%s%s ", name, kGemmTiles[s.tile].bm, kGemmTiles[s.tile].bn, s.direct ? "d" : "r",
                       s.splits > 1 ? "+" : "");
            };
            print("f", p->geo.f);
            print("dw", p->geo.dw);
            print("dx", p->geo.dx);
            printf("planes=%d\n", p->geo.dz_planes);
            wq8_linear_plan_destroy(p);
        } else {
            return 2;
        }
    }
    return 0;
}
