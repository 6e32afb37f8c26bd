// Group norm forward, x in f32.
#include "wq8_norm_fwd.h"

namespace wq8 {

wq8_status launch_norm_forward_f32(const NormGeo &g, wq8_dtype ydt, const NormPtrs &p, void *stream) {
    return norm_forward<float>(g, ydt, p, stream);
}

}  // namespace wq8
