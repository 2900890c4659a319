// gclip_rms_backward8_f16.hip -- the backward kernels of gclip_rms_backward.hpp for one storage format, with the normed
// matrix in 8 bits.
#include "gclip_rms_backward.hpp"

namespace gclip {
template hipError_t rms_backward_rows<GCLIP_F16, true>(const RmsBwdArgs&, bool, const DropArgs*, hipStream_t);
}  // namespace gclip
