// Group norm backward, x in bf16.
#include "wq8_norm_bwd.h"

namespace wq8 {

wq8_status launch_norm_backward_bf16(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream) {
    return norm_backward<bf16_t>(g, ydt, p, stream);
}

}  // namespace wq8
