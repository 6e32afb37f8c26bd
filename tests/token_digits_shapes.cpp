// Prints the launch shapes of the backward of the product of codes, one line for
// each line read:
//   rows Cin Cout x_dtype round_dz
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
    long long rows;
    int a[4];
    while (scanf("%lld %d %d %d %d", &rows, a, a + 1, a + 2, a + 3) == 5) {
        wq8_q8linear_desc d = {};
        d.rows = rows, d.Cin = a[0], d.Cout = a[1], d.x_dtype = d.y_dtype = (wq8_dtype)a[2], d.round_dz = a[3];
        wq8_q8linear_plan *p;
        if (wq8_q8linear_plan_create(&d, &p) != WQ8_OK) return 1;
        printf("planes=%d", p->geo.planes);
        const auto print = [&](const char *name, const Q8Shape &s) {
            printf(" %s=%dx%d%s", name, kQ8PairTiles[s.tile].bm, kQ8PairTiles[s.tile].bn, s.splits > 1 ? "+" : "");
        };
        print("dw", p->geo.dw);
        print("dx", p->geo.dx);
        printf("\n");
        wq8_q8linear_plan_destroy(p);
    }
    return 0;
}
