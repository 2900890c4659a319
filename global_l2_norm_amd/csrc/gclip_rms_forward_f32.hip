// gclip_rms_forward_f32.hip -- the forward kernels of gclip_rms_forward.hpp for one storage format.
#include "gclip_rms_forward.hpp"

namespace gclip {
template hipError_t rms_forward_rows<GCLIP_F32, false>(const RmsFwdArgs&, bool, const DropArgs*, hipStream_t);
}  // namespace gclip
