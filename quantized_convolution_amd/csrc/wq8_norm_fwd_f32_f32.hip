// Group norm forward, x in f32, y in f32.
#include "wq8_norm_fwd.h"

namespace wq8 {

wq8_status launch_norm_forward_f32_f32(const NormGeo &g, const NormPtrs &p, void *stream) {
    return norm_forward<float, float>(g, p, stream);
}

}  // namespace wq8
