// General forward kernel instances of the other rotary layouts, with the q/k RMSNorm.
#include "instances.cuh"

namespace qkvp {
const void* fwd_rotary_kernel_norm(const FwdVariant& v) {
  return v.head_dim == 64 ? inst::FwdPick<64, true, false, true>::pick(v)
                          : inst::FwdPick<128, true, false, true>::pick(v);
}
}  // namespace qkvp
