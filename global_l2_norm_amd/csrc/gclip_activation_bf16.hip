// gclip_activation_bf16.hip -- the kernels of gclip_activation.hpp for one storage format.
#include "gclip_activation.hpp"

namespace gclip {
template hipError_t activation_of<GCLIP_BF16>(const ActArgs&, int32_t, bool, bool, hipStream_t);
}  // namespace gclip
