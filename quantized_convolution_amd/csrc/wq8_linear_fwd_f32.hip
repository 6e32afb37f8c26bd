// Matrix product forward, x in f32.
#include "wq8_linear_fwd.h"

namespace wq8 {

wq8_status launch_linear_forward_f32(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream) {
    return linear_forward<float>(g, ydt, p, stream);
}

}  // namespace wq8
