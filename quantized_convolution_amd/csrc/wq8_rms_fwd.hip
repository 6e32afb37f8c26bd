// Root-mean-square norm forward, every pair of types.
#include "wq8_rms_fwd.h"

namespace wq8 {

wq8_status launch_rms_forward(const RowsGeo &g, wq8_dtype xdt, wq8_dtype ydt, const RmsPtrs &p, void *stream) {
    const hipStream_t st = (hipStream_t)stream;
    if (xdt == WQ8_F32) {
        if (ydt == WQ8_F32) run_rows<float, float, true>(g, p, st);
        else run_rows<float, bf16_t, true>(g, p, st);
    } else {
        if (ydt == WQ8_F32) run_rows<bf16_t, float, true>(g, p, st);
        else run_rows<bf16_t, bf16_t, true>(g, p, st);
    }
    return check_launch("root-mean-square norm");
}

}  // namespace wq8
