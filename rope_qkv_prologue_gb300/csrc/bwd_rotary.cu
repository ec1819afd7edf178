// General backward kernel instances of the other rotary layouts.
#include "instances.cuh"

namespace qkvp {
const void* bwd_rotary_kernel(const BwdVariant& v) {
  return v.norm ? inst::BwdPick<true, false, true>::pick(v) : inst::BwdPick<false, false, true>::pick(v);
}
}  // namespace qkvp
