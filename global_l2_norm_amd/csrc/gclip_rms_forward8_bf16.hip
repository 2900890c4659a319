// gclip_rms_forward8_bf16.hip -- the forward kernels of gclip_rms_forward.hpp for one storage format, with matrices in 8 bits.
#include "gclip_rms_forward.hpp"

namespace gclip {
template hipError_t rms_forward_rows<GCLIP_BF16, true>(const RmsFwdArgs&, bool, const DropArgs*, hipStream_t);
}  // namespace gclip
