// Instances of the write into the 8-bit pool: head_dim 64, without a qkv bias.
#include "pool_write8.cuh"

namespace qkvp {
const void* pool_write8_kernel_d64(int rope, bool norm) { return pool_write8_pick<64, false>(rope, norm); }
int pool_write8_smem_bytes(int head_dim, int tab_rows) {
  return kWarps * 2 * kStepBytes + tab_rows * head_dim * (int)sizeof(float);
}
int pool_write8_threads() { return 32 * kWarps; }
}  // namespace qkvp
