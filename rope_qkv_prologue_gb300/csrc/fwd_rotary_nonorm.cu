// General forward kernel instances of the other rotary layouts, without the q/k RMSNorm.
#include "instances.cuh"

namespace qkvp {
const void* fwd_rotary_kernel_nonorm(const FwdVariant& v) {
  return v.head_dim == 64 ? inst::FwdPick<64, false, false, true>::pick(v)
                          : inst::FwdPick<128, false, false, true>::pick(v);
}
}  // namespace qkvp
