// Group norm backward, x in f32.
#include "wq8_norm_bwd.h"

namespace wq8 {

wq8_status launch_norm_backward_f32(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream) {
    return norm_backward<float>(g, ydt, p, stream);
}

}  // namespace wq8
