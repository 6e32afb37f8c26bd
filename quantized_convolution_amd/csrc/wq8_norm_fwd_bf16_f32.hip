// Group norm forward, x in bf16, y in f32.
#include "wq8_norm_fwd.h"

namespace wq8 {

wq8_status launch_norm_forward_bf16_f32(const NormGeo &g, const NormPtrs &p, void *stream) {
    return norm_forward<bf16_t, float>(g, p, stream);
}

}  // namespace wq8
