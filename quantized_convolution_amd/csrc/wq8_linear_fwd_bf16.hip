// Matrix product forward, x in bf16.
#include "wq8_linear_fwd.h"

namespace wq8 {

wq8_status launch_linear_forward_bf16(const LinearGeo &g, wq8_dtype ydt, const LinearPtrs &p, void *stream) {
    return linear_forward<bf16_t>(g, ydt, p, stream);
}

}  // namespace wq8
