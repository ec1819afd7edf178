// Instances of the write into the 8-bit pool: head_dim 64, with a qkv bias.
#include "pool_write8.cuh"

namespace qkvp {
const void* pool_write8_kernel_d64_bias(int rope, bool norm) { return pool_write8_pick<64, true>(rope, norm); }
}  // namespace qkvp
