// Shared pieces of the kernels that attend single tokens over a paged pool: a warp's
// own copies into shared memory, and the walk over the concatenated tiles of all
// sequences.
#pragma once

#include "attention.cuh"

namespace qkvp {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Own keys of sequence b, within what its row of the page table can name.
__device__ __forceinline__ int dec_own(const AttnDecodeArgs& a, int b) {
  const int n = a.lengths[b], most = a.max_pages * a.page_size;
  return n < 0 ? 0 : (n > most ? most : n);
}
// Tiles of sequence b: the prefix's keys (when it is not computed apart), then its own.
__device__ __forceinline__ int dec_tiles(const AttnDecodeArgs& a, int b) {
  return (int)(((uint32_t)a.joint_len + (uint32_t)dec_own(a, b) + (uint32_t)a.tile_keys - 1) / (uint32_t)a.tile_keys);
}

// Whole warp: all tiles of the batch.
__device__ __forceinline__ int64_t dec_total(const AttnDecodeArgs& a, int lane) {
  int64_t all = 0;
#pragma unroll 8
  for (int s = lane; s < a.batch; s += 32) all += dec_tiles(a, s);
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  return all;
}

__device__ __forceinline__ int64_t dec_quota(const AttnDecodeArgs& a, int64_t total) {
  const int64_t q = (total + a.ranges - 1) / a.ranges, least = kDecMinKeys / a.tile_keys;
  return q < least ? least : q;
}

// A position in the concatenated tiles.
struct DecCursor {
  int b;      // sequence
  int tile;   // tile of it
  int tiles;  // its tiles
  // Whole warp, behind a sequence's last tile: to the next sequence that has any, 32 at a
  // time (there may be many empty ones between); past the last one it stays there, at its end.
  __device__ __forceinline__ void settle(const AttnDecodeArgs& a, int lane) {
    if (tile < tiles) return;
#pragma unroll 1
    for (int s0 = b + 1; s0 < a.batch; s0 += 32) {
      const int n = s0 + lane < a.batch ? dec_tiles(a, s0 + lane) : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
      if (some) {
        const int src = __ffs(some) - 1;
        b = s0 + src;
        tiles = __shfl_sync(0xffffffffu, n, src);
        tile = 0;
        return;
      }
    }
  }
};

// Whole warp: where tile t0 of the concatenation lies.
__device__ __forceinline__ DecCursor dec_begin(const AttnDecodeArgs& a, int64_t t0, int lane) {
  DecCursor cu{0, 0, 0};
  int64_t left = t0;
  for (int s0 = 0; s0 < a.batch; s0 += 32) {
    const int n = s0 + lane < a.batch ? dec_tiles(a, s0 + lane) : 0;
    int64_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, sum > left);
    if (past) {
      const int src = __ffs(past) - 1;
      cu.b = s0 + src;
      cu.tiles = __shfl_sync(0xffffffffu, n, src);
      cu.tile = (int)(left - (__shfl_sync(0xffffffffu, sum, src) - cu.tiles));
      break;
    }
    left -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return cu;
}

// Pool row of key `key` of sequence b, or -1 (behind its end, or a bad page).
__device__ __forceinline__ int dec_slot(const AttnDecodeArgs& a, int b, uint32_t keys, uint32_t key) {
  if (key >= keys) return -1;
  const int32_t* pages = a.prefix_pages;
  if (key >= (uint32_t)a.joint_len) {
    key -= (uint32_t)a.joint_len;
    pages = a.page_table + (int64_t)b * a.table_stride;
  }
  const uint32_t p = a.page_shift >= 0 ? key >> a.page_shift : key / (uint32_t)a.page_size;
  const int page = pages[p];
  if (page < 0 || page >= a.num_pages) {
    if (a.dev_status) atomicOr(a.dev_status, kDevBadPage);
    return -1;
  }
  return page * a.page_size + (int)(key - p * (uint32_t)a.page_size);
}

}  // namespace qkvp
