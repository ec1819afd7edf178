// Pipelined backward kernel instances of the other rotary layouts.
#include "instances.cuh"

namespace qkvp {
const void* bwd_stream_rotary_kernel(const BwdVariant& v) {
  return v.norm ? inst::BwdPick<true, true, true>::pick(v) : inst::BwdPick<false, true, true>::pick(v);
}
}  // namespace qkvp
