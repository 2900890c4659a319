// gclip_layer_backward_f32.hip -- the backward kernels of gclip_layer_backward.hpp for one storage format.
#include "gclip_layer_backward.hpp"

namespace gclip {
template hipError_t backward_rows<GCLIP_F32>(const BwdArgs&, bool, const DropArgs*, hipStream_t);
template hipError_t join_weight_grads<GCLIP_F32>(const BwdArgs&, hipStream_t);
}  // namespace gclip
