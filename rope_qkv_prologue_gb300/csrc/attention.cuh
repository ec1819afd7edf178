// Shared pieces of the attention kernels on the tensor cores (sm_103a): waits
// that give up together, tensor-memory operands, tensor-map loads of three
// dimensions, and the order in which the persistent kernels take the blocks of
// packed sequences.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "tcgen05.cuh"

namespace qkvp {

constexpr int kAttnRows = kAttnBlock;            // rows of a block (queries or keys)
constexpr int kAttnBox = kAttnRows * 128;        // bytes of 128 rows x 64 bf16, 128B-swizzled
constexpr float kLog2e = 1.4426950408889634f;

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` in a swizzled box.
__device__ __forceinline__ int attn_swz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// The kernels run long straight code in several roles at once, and at short
// sequences each role goes through all of its code for a few blocks: instruction
// fetches were a quarter of the stalls (60 sequences of 67 rows). So what is in
// many places, like a wait, is kept short.

// What the waits of a CTA watch, in shared memory.
struct __align__(8) AttnWatch {
  uint32_t fail;  // a wait gave up
  uint32_t beat;  // when this CTA last began to fetch a tile (low word of the nanosecond timer)
};
__device__ __forceinline__ uint32_t global_ns_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ void attn_beat(AttnWatch* watch) {
  *(volatile uint32_t*)&watch->beat = global_ns_lo();
}

// Bounded wait, every lane of the calling warp: with one lane polling and the
// others waiting for it, the kernels measured up to half slower. What is bounded is
// the time without progress, not the wait: some warps have nothing to do while the
// others work on a long item (the finder, the softmax of a slot that is idle), for
// seconds where a sequence has very many blocks or a group very many heads. The
// rings are a few tiles deep, so as long as anything moves the loader does. Gives up
// kWaitLimitNs after the CTA's last beat, and at once when another warp already gave
// up: after one timeout the rest of the kernel runs through without waiting, every
// loop still ends, and attn_report tells the host.
// A wait by parity sees a phase only until the next one completes. So for every
// barrier here, whatever completes phase k + 1 is behind each waiter's having seen
// phase k: a producer that could run ahead waits for something that the waiter does
// after its wait.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, AttnWatch* watch) {
  if (mbar_try_wait(bar, parity)) return true;
  uint32_t fail, beat;
  do {
    if (mbar_try_wait(bar, parity)) return true;
    asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];" : "=r"(fail), "=r"(beat) : "r"(smem_addr(watch)));
    if (fail) return false;
  } while ((int32_t)(global_ns_lo() - beat) < (int32_t)kWaitLimitNs);  // (a beat newer than the timer read is no age)
  *(volatile uint32_t*)&watch->fail = 1;
  return false;
}
static_assert(kWaitLimitNs < (1ull << 31), "the waits count nanoseconds in 32 bits");

// At the kernel's end, behind a barrier.
__device__ __forceinline__ void attn_report(const AttnWatch* watch, int* err) {
  if (threadIdx.x == 0 && *(const volatile uint32_t*)&watch->fail) atomicOr(err, kErrWaitTimeout);
}

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.b32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

// Registers per thread of this warp's group of four warps, which calls it together.
// The shares of a CTA's groups add up to no more than what it was launched with.
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A value that every lane holds, in a form the compiler knows to be uniform: the
// operands of an MMA are then computed in uniform registers, not moved there one
// by one for each MMA.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 values in a register pair, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// D[tmem] (+)= A[tmem] * B[smem]: A is M = 128 lanes x 16 bf16 per K step, two
// consecutive K values per 32-bit column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Whole warp: 16 consecutive 32-bit columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 consecutive fp32 columns of this warp's 32 TMEM lanes, in place: times f.
__device__ __forceinline__ void tmem_scale16(uint32_t addr, float f) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  tmem_st16(addr, r);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Whole warp: 64 consecutive fp32 columns, two loads and one wait. The empty asm
// keeps the uses of the second load's registers behind the wait.
__device__ __forceinline__ void tmem_ld64(uint32_t addr, float (&v)[64]) {
  uint32_t r0[32], r1[32];
  tmem_ld32_issue(addr, r0);
  tmem_ld32_issue(addr + 32, r1);
  tmem_wait_ld32(r0);
  asm volatile(""
               : "+r"(r1[0]), "+r"(r1[1]), "+r"(r1[2]), "+r"(r1[3]), "+r"(r1[4]), "+r"(r1[5]), "+r"(r1[6]), "+r"(r1[7]),
                 "+r"(r1[8]), "+r"(r1[9]), "+r"(r1[10]), "+r"(r1[11]), "+r"(r1[12]), "+r"(r1[13]), "+r"(r1[14]),
                 "+r"(r1[15]), "+r"(r1[16]), "+r"(r1[17]), "+r"(r1[18]), "+r"(r1[19]), "+r"(r1[20]), "+r"(r1[21]),
                 "+r"(r1[22]), "+r"(r1[23]), "+r"(r1[24]), "+r"(r1[25]), "+r"(r1[26]), "+r"(r1[27]), "+r"(r1[28]),
                 "+r"(r1[29]), "+r"(r1[30]), "+r"(r1[31]));
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = __uint_as_float(r0[i]);
    v[32 + i] = __uint_as_float(r1[i]);
  }
}

// The maximum of 32 values, in two chains of three-input maxima.
__device__ __forceinline__ float max32(const float* v) {
  float a = max3(v[0], v[1], v[2]), b = max3(v[3], v[4], v[5]);
#pragma unroll
  for (int i = 6; i < 30; i += 4) {
    a = max3(a, v[i], v[i + 1]);
    b = max3(b, v[i + 2], v[i + 3]);
  }
  a = max3(a, v[30], v[31]);
  return fmaxf(a, b);
}

// Whole warp: 128 consecutive fp32 columns of this warp's 32 TMEM lanes into v, and
// their maximum: a quarter's maximum is taken while the next quarter loads.
__device__ __forceinline__ float tmem_ld128_max(uint32_t addr, float (&v)[128]) {
  uint32_t r0[32], r1[32], r2[32], r3[32];
  auto keep = [&](const uint32_t (&r)[32], int x) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[32 * x + i] = __uint_as_float(r[i]);
  };
  tmem_ld32_issue(addr, r0);
  tmem_wait_ld32(r0);
  tmem_ld32_issue(addr + 32, r1);
  keep(r0, 0);
  const float m0 = max32(v);
  tmem_wait_ld32(r1);
  tmem_ld32_issue(addr + 64, r2);
  keep(r1, 1);
  const float m1 = max32(v + 32);
  tmem_wait_ld32(r2);
  tmem_ld32_issue(addr + 96, r3);
  keep(r2, 2);
  const float m2 = max32(v + 64);
  tmem_wait_ld32(r3);
  keep(r3, 3);
  return fmaxf(max3(m0, m1, m2), max32(v + 96));
}

// 3-D tensor-map load (c0: the contiguous coordinate).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}

// D = A B^T over K = HD, both operands K-major boxes of 64 columns. The whole warp
// calls it (and attn_mma_ts) with uniform operands; one elected lane issues.
template <int HD>
__device__ __forceinline__ void attn_mma_ss(uint32_t d, const unsigned char* a, const unsigned char* b, uint32_t id) {
  const uint64_t ad = umma_desc_sw128(a), bd = umma_desc_sw128(b);
  if (elect_one()) {
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
      const int off = (k >> 2) * (kAttnBox >> 4) + 2 * (k & 3);
      umma_bf16(d, ad + off, bd + off, id, k != 0);
    }
  }
}

// D (+)= W B over the 128 keys or queries of a block: W bf16 in tensor memory, the
// K steps of its second half `half` columns behind the first's; B read MN-major.
__device__ __forceinline__ void attn_mma_ts(uint32_t d, uint32_t w, int half, const unsigned char* b, uint32_t id,
                                            bool more) {
  const uint64_t bd = umma_desc_sw128_mn(b, kAttnBox);
  if (elect_one()) {
#pragma unroll
    for (int k = 0; k < kAttnRows / 16; ++k)
      umma_bf16_ts(d, w + half * (k >> 2) + 8 * (k & 3), bd + 128 * k, id, more || k != 0);
  }
}

// Whole warp, lanes taking copies in turn: a tile of 128 rows of q or dout. With hs = 2
// it is 128 rows of one head (`map`); for short sequences it has four pieces of 32 rows
// (`pieces`, a box of 32): with hs = 1 the 64 rows of two heads, with hs = 0 the 32 rows of
// four; piece p is the rows 32 (p mod 2^hs) .. of head p / 2^hs, from (col, row) on.
template <int HD>
__device__ __forceinline__ void attn_load_tile(unsigned char* dst, const CUtensorMap* map, const CUtensorMap* pieces,
                                               int col, int row, int hs, uint64_t* bar, int lane) {
  constexpr int X = HD / 64;
  const int x = lane % X, p = lane / X;
  if (hs == 2) {
    if (p == 0) tma_load_2d(dst + x * kAttnBox, map, col + 64 * x, row, bar);
  } else if (p < 4) {
    tma_load_2d(dst + x * kAttnBox + p * (kAttnBox / 4), pieces, col + (p >> hs) * HD + 64 * x,
                row + 32 * (p & ((1 << hs) - 1)), bar);
  }
}

// The blocks of packed sequences, taken from the most expensive to the cheapest.
// Sequence s has n_s = ceil(len_s / unit) blocks, one of each cost 1 .. n_s (with the
// causal mask the block at distance c from the sequence's beginning, or end, has c times
// the work of the first). Classes of costs (lo, hi] follow each other downwards from the
// largest n_s, single costs up to 15 and an eighth wide above; in a class the sequences
// follow in their order, each with min(n_s, hi) - lo blocks. Evaluated by one warp from
// the sequence offsets alone: no list in memory, no launch before the kernel that uses it.
//
// The work items of a CTA ascend, so the finder keeps its place, a class and a group of
// 32 sequences in it, and only goes on from there: each class is gone through twice (its
// size, then its items), whatever the number of items. With a search through all sequences
// for every item, 32768 sequences of 70 rows, 2 over 2 heads of 64, took 231 ms instead
// of 2.3.
//
// Every block is `units` work items (heads, pairs of heads, ...). Short sequences
// come last and have counts of their own, since one tile of 128 rows holds several
// heads of them: units64 for those of at most 64 rows (two heads to a tile) and
// units32 for those of at most 32 (four); 0 where the caller has no use for that.
struct AttnOrder {
  static constexpr int kCached = 128;  // sequences whose block counts are kept in shared memory
  const int32_t* cu;
  int batch;
  int unit;
  uint32_t units, units64, units32;
  int* cache;      // [kCached]
  uint32_t total;  // sum of n_s
  uint32_t n64, n32;
  // the place of the finder
  int cls;               // 2: the class (lo, hi]; 1, 0: the short sequences, as hs in attn_load_tile
  int lo, hi;
  uint32_t first, size;  // rank of the class's first block, and its blocks
  int s0;                // the next 32 sequences to look at
  uint32_t before;       // blocks of the class in the sequences before them

  // n_s, or -1 (one of n64) or -2 (of n32)
  __device__ __forceinline__ int count(int64_t rows) const {
    if (units64 && rows <= 64 && rows > 0) return rows <= 32 ? -2 : -1;
    return (int)((rows + unit - 1) / unit);
  }
  __device__ __forceinline__ int blocks(int s) const {
    return s < kCached ? cache[s] : count((int64_t)cu[s + 1] - cu[s]);
  }
  // Blocks of sequence s that belong to the class.
  __device__ __forceinline__ uint32_t members(int s) const {
    if (s >= batch) return 0;
    const int n = blocks(s);
    return cls == 2 ? (uint32_t)max(min(n, hi) - lo, 0) : (uint32_t)(n == cls - 2);
  }

  // Whole warp. False (and no blocks) when the offsets do not ascend in [0, T].
  __device__ __forceinline__ bool init(int64_t T, int lane) {
    bool bad = false;
    uint32_t sum = 0, top = 0, a64 = 0, a32 = 0;
#pragma unroll 1  // (code size, here and below)
    for (int s = lane; s < batch; s += 32) {
      const int64_t a = cu[s], b = cu[s + 1];
      const bool ok = a >= 0 && b >= a && b <= T;
      bad |= !ok;
      const int n = ok ? count(b - a) : 0;
      if (s < kCached) cache[s] = n;
      a64 += n == -1;
      a32 += n == -2;
      sum += max(n, 0);
      top = max((int)top, n);
    }
    bad = __any_sync(0xffffffffu, bad);
    total = bad ? 0u : __reduce_add_sync(0xffffffffu, sum);
    n64 = bad ? 0u : __reduce_add_sync(0xffffffffu, a64);
    n32 = bad ? 0u : __reduce_add_sync(0xffffffffu, a32);
    cls = 2;
    lo = hi = bad ? 0 : (int)__reduce_max_sync(0xffffffffu, top);  // an empty class above the first
    first = size = before = 0;
    s0 = 0;
    __syncwarp();
    return !bad;
  }

  __device__ __forceinline__ uint32_t work() const { return total * units + n64 * units64 + n32 * units32; }

  // Whole warp: work item w < work() is unit `unit_of` of the block of cost `cost` of
  // sequence `seq`; hs as in attn_load_tile. w is larger than in the call before.
  __device__ __forceinline__ void find(uint32_t w, int lane, int& seq, int& cost, int& unit_of, int& hs) {
    const uint32_t w0 = total * units, w1 = w0 + n64 * units64;
    hs = w < w0 ? 2 : (w < w1 ? 1 : 0);
    const uint32_t at = w - (hs == 2 ? 0u : (hs == 1 ? w0 : w1)), per = hs == 2 ? units : (hs == 1 ? units64 : units32);
    const uint32_t r = at / per;
    unit_of = (int)(at - r * per);
    if (hs != cls) {
      cls = hs;
      first = before = 0;
      s0 = 0;
    }
#pragma unroll 1
    while (hs == 2 && r - first >= size && lo > 0) {
      first += size;
      hi = lo;
      lo = hi - max(hi >> 3, 1);
      size = before = 0;
      uint32_t from = 0x7fffffffu;  // the class's first sequence
#pragma unroll 1
      for (int s = lane; s < batch; s += 32) {
        const uint32_t m = members(s);
        size += m;
        from = min(from, m ? (uint32_t)s : 0x7fffffffu);
      }
      size = __reduce_add_sync(0xffffffffu, size);
      s0 = size ? (int)__reduce_min_sync(0xffffffffu, from) & ~31 : 0;
    }
    uint32_t idx = r - first - before, m, here;
#pragma unroll 1
    for (;;) {
      m = members(s0 + lane);
      here = __reduce_add_sync(0xffffffffu, m);
      if (idx < here || s0 + 32 >= batch) break;
      idx -= here;
      before += here;
      s0 += 32;
    }
    uint32_t upto = m;  // of the class in the sequences s0 .. s0 + lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const int src = (__ffs(__ballot_sync(0xffffffffu, upto > idx)) - 1) & 31;
    seq = min(s0 + src, batch - 1);
    // the block's place among the m of its sequence, the dearest first
    const uint32_t into = idx - (__shfl_sync(0xffffffffu, upto, src) - __shfl_sync(0xffffffffu, m, src));
    cost = hs == 2 ? lo + (int)(__shfl_sync(0xffffffffu, m, src) - into) : 1;
  }
};

// Work item of round k for CTA b of g: the items descend in cost, and every
// other round is dealt backwards, so that the sums stay even.
__device__ __forceinline__ uint32_t attn_deal(uint32_t k, uint32_t b, uint32_t g) {
  return k * g + ((k & 1) ? g - 1 - b : b);
}

// Rows of no sequence ([0, first) and [last, T)): `chunks` 16-byte pieces per row
// set to zero, one warp of each CTA.
__device__ __forceinline__ void attn_zero_rows(uint4* out, int64_t T, int chunks, int64_t first, int64_t last,
                                               int lane) {
#pragma unroll 1
  for (int64_t r = blockIdx.x; r < first + T - last; r += gridDim.x) {
    uint4* row = out + (r < first ? r : last + (r - first)) * chunks;
#pragma unroll 1
    for (int c = lane; c < chunks; c += 32) row[c] = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace qkvp
