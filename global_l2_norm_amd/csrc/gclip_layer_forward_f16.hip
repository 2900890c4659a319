// gclip_layer_forward_f16.hip -- the forward kernels of gclip_layer_forward.hpp for one storage format.
#include "gclip_layer_forward.hpp"

namespace gclip {
template hipError_t forward_rows<GCLIP_F16>(const FwdArgs&, bool, const DropArgs*, hipStream_t);
}  // namespace gclip
