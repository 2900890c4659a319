// gclip_layer_forward_f32.hip -- the forward kernels of gclip_layer_forward.hpp for one storage format.
#include "gclip_layer_forward.hpp"

namespace gclip {
template hipError_t forward_rows<GCLIP_F32>(const FwdArgs&, bool, const DropArgs*, hipStream_t);
}  // namespace gclip
