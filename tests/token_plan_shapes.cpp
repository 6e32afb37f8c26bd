// Prints the launch shapes that plans of the operators on 8-bit codes choose, one
// line for each line read:
//   q8linear rows Cin Cout x_dtype
//   rows rows C
// Built by the host tests from the plans' own source; launches are left out.
#include <stdio.h>

#include "../quantized_convolution_amd/csrc/wq8_token_plan.cpp"

namespace wq8 {
wq8_status fail(wq8_status st, const char *, ...) { return st; }
void clear_error() {}
wq8_status launch_rms_forward(const RowsGeo &, wq8_dtype, wq8_dtype, const RmsPtrs &, void *) { return WQ8_OK; }
wq8_status launch_rms_backward(const RowsGeo &, wq8_dtype, wq8_dtype, const RmsPtrs &, void *) { return WQ8_OK; }
wq8_status launch_pack_rows(const RowsGeo &, wq8_dtype, const void *, int8_t *, float *, void *) { return WQ8_OK; }
wq8_status launch_pack_groups(const RowsGeo &, wq8_dtype, const void *, int8_t *, float *, void *) { return WQ8_OK; }
wq8_status launch_unpack(const RowsGeo &, wq8_dtype, const int8_t *, const float *, void *, void *) { return WQ8_OK; }
wq8_status launch_q8_forward(const Q8Geo &, wq8_dtype, const Q8Ptrs &, void *) { return WQ8_OK; }
wq8_status launch_q8_backward(const Q8Geo &, wq8_dtype, wq8_dtype, const Q8Ptrs &, void *) { return WQ8_OK; }
}  // namespace wq8

int main() {
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        long long rows;
        int a[3];
        if (sscanf(line, "q8linear %lld %d %d %d", &rows, a, a + 1, a + 2) == 4) {
            const wq8_q8linear_desc d = {rows, a[0], a[1], WQ8_ACT_GELU, (wq8_dtype)a[2], (wq8_dtype)a[2], WQ8_NHWC, 0, 0, 0, 0};
            wq8_q8linear_plan *p;
            if (wq8_q8linear_plan_create(&d, &p) != WQ8_OK) return 1;
            const auto print = [&](const char *name, const Q8Tile *t, const Q8Shape &s) {
                if (s.tile < 0) printf("%s=%s ", name, s.tile != kQ8Thin ? "rows" : rows <= 16 ? "thin16" : "thin32");
                else printf("%s=%dx%d%s ", name, t[s.tile].bm, t[s.tile].bn, s.splits > 1 ? "+" : "");
            };
            print("f", kQ8Tiles, p->geo.f);
            print("dw", kQ8PairTiles, p->geo.dw);
            print("dx", kQ8PairTiles, p->geo.dx);
            printf("\n");
            wq8_q8linear_plan_destroy(p);
        } else if (sscanf(line, "rows %lld %d", &rows, a) == 2) {
            const wq8_rms_desc d = {rows, a[0], 1e-6f, WQ8_BF16, WQ8_BF16, 0, 0};
            wq8_rms_plan *p;
            if (wq8_rms_plan_create(&d, &p) != WQ8_OK) return 1;
            printf("f=%dx%d b=%dx%d\n", p->f.s.lanes, p->f.s.unroll, p->b.s.lanes, p->b.s.unroll);
            wq8_rms_plan_destroy(p);
        } else {
            return 2;
        }
    }
    return 0;
}
