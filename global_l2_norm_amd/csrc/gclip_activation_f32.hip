// gclip_activation_f32.hip -- the kernels of gclip_activation.hpp for one storage format.
#include "gclip_activation.hpp"

namespace gclip {
template hipError_t activation_of<GCLIP_F32>(const ActArgs&, int32_t, bool, bool, hipStream_t);
}  // namespace gclip
