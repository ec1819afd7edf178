// Attention of one new token per sequence over the paged pool in 8 bits, split over the
// keys: the walk, the split and the join are those of attention_decode.cu.
//
// With codes K, V and scales a_j, b_j of key j's blocks (float32),
//     t_j = c a_j q . K_j,   l = sum_j 2^(t_j - m),         max t_j - 15 <= m <= max t_j - 11,
//     u_j = t_j + log2(b_j), O = sum_j 2^(u_j - n) V_j,     max u_j - 15 <= n <= max u_j - 11,
//     out = 2^r O / l,       r = n - m
// (m is a float32, whose steps from 2^27 on are 16 and more: t_j - m is then 0 or 16. r is what
// is kept, since such an m and n may differ by less than a step):
// the value scale is part of the weight, and the weights have a reference of their own,
// so their 11 significant bits are those of the largest contributions however far apart
// the blocks' scales are. The largest weight is 2^11 to 2^15, near the end of f16's range:
// one loses bits only 2^-25 below it, and vanishes 2^-36 below it (with weights of at most 1
// a key that takes nearly all the weight, its value near 0, left nothing of the others). A
// partial result leaves as (z, 2^w, 2^w 2^r O / l), z = m + log2 l rounded and w what its
// rounding left, which joins as plain softmax's do.
//
// Codes go to the matrix units (m16n8k16, f16 with fp32 accumulation) as f16, which
// holds every e4m3 value exactly; one conversion instruction makes two values. A row of
// q is scaled by a power of two that brings its largest magnitude into [2^15, 2^16), the end of
// f16's range, so that values down to 2^-32 of it keep all their bits (a channel far above the
// others may meet keys that have nothing in it). The heads
// are the products' 8 columns (S^T = K Q^T, O^T = V^T W^T): keys and values fill the 16
// rows, where heads as rows left half of them empty in groups of up to 8, at 32 products
// and 570 instructions a tile of 32 keys and 64 values instead of 16 and 440. The order of
// d in K Q^T is free: a lane's four consecutive codes are two operand registers of one
// step, so ldmatrix on bytes needs no shuffling. For V^T W^T the transposing ldmatrix moves
// pairs of codes (d, d + 1) of two keys; a byte permutation makes the pairs of keys of d and
// of d + 1, which are rows g and g + 8. The weights turn from keys by heads to heads by keys
// with a matrix move per 8 keys.
//
// Bound by the codes' bytes in long batches, where both kernels take (32 over 8 heads of
// 128, up to 32768 keys) 230 us for 48 sequences, 6.71 TB/s or 0.99 of a plain copy's rate
// (heads as rows: 253 us). 256 sequences of up to 4096 keys, 64 over 8 heads of 64: 115 to 119
// us, 5.05 TB/s (132 us): 55 % of the issue slots, and the join is a tenth. Over 4 heads 89 us
// (X = 2: twice the softmax arithmetic a byte, 56 % of the slots of 12 warps). One sequence of
// 131072 keys: 55 us (58 us), a dozen of them the start, the last tiles and the join.
#include <cuda_fp16.h>

#include "attention_decode.cuh"
#include "e4m3.cuh"

namespace qkvp {
namespace {

template <int HD, int X>
struct Dec8Shape {
  static constexpr int kKeys = kDec8Keys;
  static constexpr int kTileBytes = 2 * kKeys * HD;  // k codes, then v codes
  static constexpr int kStages = 3;
  static constexpr int kWarps = dec8_warps(HD, X == 2);  // at most 192 KiB an SM
  static constexpr int kWarpBytes = kStages * kTileBytes;
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void mma16816h(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values over the warp, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Maximum over the eight lanes of a head.
__device__ __forceinline__ float head_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The largest factor of a product q . K. With q in 16 bits (128 values below 2^16) and codes
// below 2^9 such a product is below 2^32, so scores stay below 2^99 and no infinities meet. A
// larger factor is taken as this one: what is lost is the order among keys whose scores are all
// 2^34 and more (the least product that is not 0 is 2^-33).
constexpr float kFactorMost = 0x1p67f;
// A head's reference before its first key: so low that any score passes it.
constexpr float kNoKey = -1e30f;
// Powers of two by which the largest score lies above a head's reference: when that is set,
// and where it has to move.
constexpr float kAbove = 11.f, kAboveMost = 15.f;

// Place of 16-byte chunk ch of a tile's row, so that the 8 rows of a matrix of ldmatrix
// lie in different banks: rows of 128 bytes, or of 64 (two to a line).
template <int HD>
__device__ __forceinline__ int dec8_at(int row, int ch) {
  return row * HD + ((HD == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) << 4);
}

}  // namespace

// X: groups of 8 query heads that a warp's products hold (1 or 2).
template <int HD, int X>
__global__ void __launch_bounds__(32 * dec8_warps(HD, X == 2), 1) qkvp_attention_decode8_kernel(const AttnDecodeArgs a) {
  using SH = Dec8Shape<HD, X>;
  constexpr int ST = SH::kStages, KT = SH::kKeys, NT = KT / 8, kDec8Warps = SH::kWarps;
  constexpr int CH = HD / 16, RPI = 32 / CH;  // 16-byte chunks per row, rows per copy instruction
  static_assert(KT == 32, "a lane per key");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint32_t s_in[kDec8Warps][ST];          // bit i: key i of the stage's tile is attended
  __shared__ float s_scale[kDec8Warps][ST][2][KT];   // its keys' scales as they are stored
  __shared__ float2 s_key[kDec8Warps][KT];           // a, log2 b of the tile at work
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_addr(smem_raw) + warp * SH::kWarpBytes;
  griddep_wait();
  griddep_launch_dependents();

  const int64_t total = dec_total(a, lane);
  const int64_t quota = dec_quota(a, total);
  const int heads = a.n_kv * a.head_blocks;
  const int items = a.ranges * heads;
  for (int w = blockIdx.x * kDec8Warps + warp; w < items; w += gridDim.x * kDec8Warps) {
    const int range = w / heads;
    const int64_t t0 = range * quota;
    if (t0 >= total) break;
    const int n_tiles = (int)min(quota, total - t0);
    const int hv = w % heads, kvh = hv / a.head_blocks, hb = hv % a.head_blocks;
    const int head0 = kvh * a.group + hb * 8 * X, n_heads = min(8 * X, a.group - hb * 8 * X);
    DecCursor cu = dec_begin(a, t0, lane);  // where the range begins

    // Loads run ST - 1 tiles ahead of the arithmetic, and the page lookup of a
    // tile one step ahead of its loads.
    DecCursor ld = cu;
    uint32_t ld_keys = (uint32_t)dec_own(a, ld.b);
    int slot = -1;
    auto look_up = [&]() { slot = dec_slot(a, ld.b, ld_keys, (uint32_t)(ld.tile * KT + lane)); };
    auto advance = [&]() {
      if (++ld.tile < ld.tiles) return;
      ld.settle(a, lane);
      ld_keys = (uint32_t)dec_own(a, ld.b);
    };
    const int ch = lane % CH, row_ch = a.n_kv * CH;
    const uint32_t lane_to = dec8_at<HD>(lane / CH, ch);  // (its place in the rows RPI i .. of a tile, or with bit 6 turned)
    const uint4* k_src = a.k_pool + kvh * CH + ch;
    const uint4* v_src = a.v_pool + kvh * CH + ch;
    auto issue = [&](uint32_t st) {
      const uint32_t in = __ballot_sync(0xffffffffu, slot >= 0);
      if (lane == 0) s_in[warp][st] = in;
      const uint32_t mine = (uint32_t)max(slot, 0);
      const int64_t at = (int64_t)(a.block_shift >= 0 ? mine >> a.block_shift : mine / (uint32_t)a.block) * a.n_kv + kvh;
      cp_async4(smem_addr(&s_scale[warp][st][0][lane]), a.k_scale + at, slot >= 0);
      cp_async4(smem_addr(&s_scale[warp][st][1][lane]), a.v_scale + at, slot >= 0);
      const uint32_t dst = ring + st * SH::kTileBytes;
#pragma unroll
      for (int i = 0; i < KT / RPI; ++i) {
        const int row = __shfl_sync(0xffffffffu, slot, i * RPI + lane / CH);
        const int64_t off = (int64_t)max(row, 0) * row_ch;
        const uint32_t to = dst + i * RPI * HD + ((i * RPI) & 4 ? lane_to ^ 64 : lane_to);
        cp_async16(to, k_src + off, row >= 0);
        cp_async16(to + KT * HD, v_src + off, row >= 0);
      }
    };
    look_up();
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      if (i < n_tiles) {
        issue(i);
        if (i + 1 < n_tiles) {
          advance();
          look_up();
        }
      }
      cp_commit();
    }

    // A lane has the heads 8 x + 2 (lane % 4) + y of products, and of each the keys lane / 4 + 8 i
    // of scores and the values 16 j + 2 (lane / 4), + 1 of results: o[j][x][y], o[j][x][2 + y].
    uint32_t qf[HD / 16][2 * X];
    float o[HD / 16][X][4], m[X][2], rel[X][2], l[X][2], c[X][2];  // rel: n - m; c: a head's factor
    auto begin = [&]() {                                        // a sequence's first tile here
#pragma unroll
      for (int x = 0; x < X; ++x) {
        const int r = (lane >> 2) + 8 * x;
        const uint2* src = reinterpret_cast<const uint2*>(a.q + ((int64_t)cu.b * a.n_q + head0 + r) * HD) + (lane & 3);
        uint2 raw[HD / 16];
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          raw[ks] = r < n_heads ? src[4 * ks] : make_uint2(0, 0);
          top = max(max(top, (raw[ks].x << 16) & 0x7fffffffu), max(raw[ks].x & 0x7fffffffu, raw[ks].y & 0x7fffffffu));
          top = max(top, (raw[ks].y << 16) & 0x7fffffffu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e, which brings the largest magnitude into [2^15, 2^16) (within what float32 can
        // scale by: a row below 2^-111 stays below that, with all its bits)
        const int e = min(max((int)(top >> 23) - 127 - 15, -126), 112);
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        const float factor = a.scale_log2 * __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          c[x][y] = __shfl_sync(0xffffffffu, factor, 8 * (lane & 3) + 4 * y);
          m[x][y] = kNoKey;
          rel[x][y] = l[x][y] = 0.f;
        }
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          qf[ks][x] = pack_h2(__uint_as_float(raw[ks].x << 16) * f, __uint_as_float(raw[ks].x & 0xffff0000u) * f);
          qf[ks][X + x] = pack_h2(__uint_as_float(raw[ks].y << 16) * f, __uint_as_float(raw[ks].y & 0xffff0000u) * f);
        }
      }
#pragma unroll
      for (int j = 0; j < HD / 16; ++j)
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[j][x][y] = 0.f;
    };
    bool first = cu.tile == 0;  // of the sequence: else the segment continues one of the range before
    auto end = [&]() {          // its last tile here: the partial result
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float sum = l[x][y];
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
          const int h = 8 * x + 2 * (lane & 3) + y;
          if (h < n_heads) {
            const int64_t row = (int64_t)(first ? cu.b : a.batch + range) * a.n_q + head0 + h;
            // what ref's rounding takes from log2 l, or adds to it, goes into the sum and the result
            const float ls = __log2f(sum), ref = m[x][y] + ls, rest = ex2((m[x][y] - ref) + ls);
            // (two factors: their product may be too small for a float where the result is not)
            const float f = sum == 0.f ? 0.f : __fdividef(rest, sum), e = ex2(rel[x][y]);
            if ((lane >> 2) == 0) a.part_ml[row] = sum == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(ref, rest);
            float2* dst = reinterpret_cast<float2*>(a.part_o + row * HD) + (lane >> 2);
#pragma unroll
            for (int j = 0; j < HD / 16; ++j) dst[8 * j] = make_float2(f * o[j][x][y] * e, f * o[j][x][2 + y] * e);
          }
        }
    };
    begin();
    uint32_t st = 0;
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      cp_wait<ST - 2>();
      __syncwarp();  // this tile is here, and every lane is done with the one before
      if (t + ST - 1 < n_tiles) {
        issue(st == 0 ? ST - 1 : st - 1);
        if (t + ST < n_tiles) {
          advance();
          look_up();
        }
      }
      cp_commit();
      const uint32_t in = s_in[warp][st];
      s_key[warp][lane] =
          make_float2(clamp_scale(s_scale[warp][st][0][lane]), __log2f(clamp_scale(s_scale[warp][st][1][lane])));
      const uint32_t kt = ring + st * SH::kTileBytes, vt = kt + KT * HD;
      float s[NT / 2][X][4];  // [y]: key lane / 4 of 16; [2 + y]: 8 behind it
#pragma unroll
      for (int i = 0; i < NT / 2; ++i)
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[i][x][y] = 0.f;
#pragma unroll
      for (int i = 0; i < NT / 2; ++i)
#pragma unroll
        for (int k4 = 0; k4 < HD / 64; ++k4) {
          uint32_t b[2][4];
#pragma unroll
          for (int v = 0; v < 2; ++v)
            ldsm4(kt + dec8_at<HD>(16 * i + 8 * v + (lane & 7), 4 * k4 + (lane >> 3)), b[v]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a0, a1, a2, a3;
            from_e4m3x4(b[0][k], a0, a2);
            from_e4m3x4(b[1][k], a1, a3);
#pragma unroll
            for (int x = 0; x < X; ++x) mma16816h(s[i][x], a0, a1, a2, a3, qf[4 * k4 + k][x], qf[4 * k4 + k][X + x]);
          }
        }
      __syncwarp();  // s_key is written
      float2 key[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) key[i] = s_key[warp][8 * i + (lane >> 2)];
      float d[NT][X][2], e[NT][X][2];  // t - m and u - n
      // t is rounded before m is taken from it: m is a rounded score less a little, and with the
      // unrounded one the difference would hold what its rounding left, 2^3 and more for
      // scores from 2^27 on. bound: whether factors may lie above theirs.
      auto factor = [&](int i, int x, int y, bool bound) {
        const float f = key[i].x * c[x][y];
        return bound ? fminf(f, kFactorMost) : f;
      };
      auto exponents = [&](bool bound) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)  // (packed, the two operations become one)
              d[i][x][y] = __fsub_rn(__fmul_rn(s[i >> 1][x][2 * (i & 1) + y], factor(i, x, y, bound)), m[x][y]);
        if (in != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (!((in >> (8 * i + (lane >> 2))) & 1)) {
#pragma unroll
              for (int x = 0; x < X; ++x) d[i][x][0] = d[i][x][1] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < X; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              e[i][x][y] = d[i][x][y] + (key[i].y - rel[x][y]);
              top = max3(top, d[i][x][y], e[i][x][y]);
            }
        return top;
      };
      // A head's references only move where a score passes them by too much; until then no
      // lane has to know the others' maxima. (Factors above their bound come this way too.)
      float a_most = key[0].x, c_most = c[0][0];
#pragma unroll
      for (int i = 1; i < NT; ++i) a_most = fmaxf(a_most, key[i].x);
#pragma unroll
      for (int x = 0; x < X; ++x) c_most = max3(c_most, c[x][0], c[x][1]);
      if (__any_sync(0xffffffffu, exponents(false) > kAboveMost || a_most * c_most > kFactorMost)) {
        auto score = [&](int i, int x, int y) { return __fmul_rn(s[i >> 1][x][2 * (i & 1) + y], factor(i, x, y, true)); };
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if ((in >> (8 * i + (lane >> 2))) & 1) top = fmaxf(top, score(i, x, y));
            const float m_new = fmaxf(m[x][y], head_max(top) - kAbove), down = m[x][y] - m_new;
            float tow = -INFINITY;  // of u - m
#pragma unroll
            for (int i = 0; i < NT; ++i)
              if ((in >> (8 * i + (lane >> 2))) & 1) tow = fmaxf(tow, (score(i, x, y) - m_new) + key[i].y);
            const float rel_new = fmaxf(rel[x][y] + down, head_max(tow) - kAbove);
            l[x][y] *= ex2(down);
            const float f = ex2(rel[x][y] + down - rel_new);
            m[x][y] = m_new;
            rel[x][y] = rel_new;
#pragma unroll
            for (int j = 0; j < HD / 16; ++j) {
              o[j][x][y] *= f;
              o[j][x][2 + y] *= f;
            }
          }
        exponents(true);
      }
      uint32_t pf[NT][X];  // the weights as the second product's operand: a head's keys
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < X; ++x) {
#pragma unroll
          for (int y = 0; y < 2; ++y) l[x][y] += ex2(d[i][x][y]);
          pf[i][x] = transposed(pack_h2(ex2(e[i][x][0]), ex2(e[i][x][1])));
        }
      {
        const int row = (((lane >> 3) & 1) << 3) + (lane & 7), hi = lane >> 4;
#pragma unroll
        for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
          for (int j = 0; j < HD / 16; j += 2) {
            uint32_t b[4], e0, o0, e1, o1;
            ldsm4t(vt + dec8_at<HD>(16 * k2 + row, j + hi), b);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              from_e4m3x4(__byte_perm(b[2 * i], 0, 0x3120), e0, o0);
              from_e4m3x4(__byte_perm(b[2 * i + 1], 0, 0x3120), e1, o1);
#pragma unroll
              for (int x = 0; x < X; ++x) mma16816h(o[j + i][x], e0, o0, e1, o1, pf[2 * k2][x], pf[2 * k2 + 1][x]);
            }
          }
      }
      st = st + 1 == ST ? 0 : st + 1;
      // the ranges that a sequence begins and ends in, for the joining kernel
      if (hv == 0 && lane == 0) {
        if (cu.tile == 0) a.plan[cu.b].x = range;
        if (cu.tile + 1 == cu.tiles) a.plan[cu.b].y = range;
      }
      if (++cu.tile == cu.tiles || t + 1 == n_tiles) {
        end();
        cu.settle(a, lane);
        first = true;
        if (t + 1 < n_tiles) begin();
      }
    }
    cp_wait<0>();
    __syncwarp();
  }
}

const void* attention_decode8_kernel(int head_dim, bool wide) {
  if (head_dim == 64)
    return wide ? reinterpret_cast<const void*>(&qkvp_attention_decode8_kernel<64, 2>)
                : reinterpret_cast<const void*>(&qkvp_attention_decode8_kernel<64, 1>);
  return wide ? reinterpret_cast<const void*>(&qkvp_attention_decode8_kernel<128, 2>)
              : reinterpret_cast<const void*>(&qkvp_attention_decode8_kernel<128, 1>);
}
int attention_decode8_smem_bytes(int head_dim, bool wide) {
  return dec8_warps(head_dim, wide) * (head_dim == 64 ? Dec8Shape<64, 1>::kWarpBytes : Dec8Shape<128, 1>::kWarpBytes);
}

}  // namespace qkvp
