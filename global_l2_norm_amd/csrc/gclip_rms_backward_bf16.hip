// gclip_rms_backward_bf16.hip -- the backward kernels of gclip_rms_backward.hpp for one storage format.
#include "gclip_rms_backward.hpp"

namespace gclip {
template hipError_t rms_backward_rows<GCLIP_BF16, false>(const RmsBwdArgs&, bool, const DropArgs*, hipStream_t);
template hipError_t rms_join_weight_grad<GCLIP_BF16>(const RmsBwdArgs&, hipStream_t);
}  // namespace gclip
