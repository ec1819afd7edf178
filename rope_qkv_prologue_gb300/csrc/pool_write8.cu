// The prologue of new tokens with the keys and values going into a paged pool in 8
// bits: e4m3 codes and a scale for each block of `block` tokens and head.
//
// With x a head's row (k normed and rotated, v as it is) in float32 and amax the
// largest magnitude that this call writes into a block, the block's scale is
//     s = max(amax / 448, 2^-100)   where the call writes the block's first token,
//     s = s_old 2^k, k >= 0 least with amax <= 448 s   where earlier tokens are held;
// a code is rne(x / s), and with k > 0 the held codes are divided by 2^k. Powers of two
// only: a held code then loses bits only where it falls below e4m3's normal range,
// so that a block which grows token by token is not rounded anew each time. A code's
// error is half a step of e4m3, 2^-4 of the value (2^-10 s below 2^-6 s): with a
// floating code the scale has to keep the values in range, not to centre them.
//
// Work. A CTA takes `tile` tokens. The tokens of one block that follow each other are a
// run; the CTA whose tile has a run's first token does the whole run. A warp takes one
// (run, head, k or v) at a time, tokens side by side (a row of a head is CPH / 2 lanes, two
// chunks of 8 values each: the units of rot_unit), so amax is a maximum over registers and
// lanes and the codes are formed from registers: the row is read once. Runs of more than
// kHold passes are read twice (the second time from L2). Query heads are the same without
// a block, kQueryRows rows of a lane in flight at once.
//
// cos and sin of the tile's tokens are computed once per CTA into shared memory, for all
// its heads; tokens of a run beyond the table's end get theirs computed by the lanes
// that use them.
#include <cuda_fp16.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "qkv_prologue.h"

namespace qkvp {
namespace {

constexpr int kWarps = 8;
constexpr int kHold = 4;       // passes of a run whose values stay in registers
constexpr int kQueryRows = 4;  // rows of query heads in flight per lane

struct Row {
  float2 lo[4], hi[4];
};

template <int HD>
struct Tile {
  static constexpr int CPH = HD / 8, PPH = CPH / 2, HALF = HD / 2;
  static constexpr int ROWS = 32 / PPH;  // rows of a head that a warp holds at once
};

// Position of a head in the packed row.
__device__ __forceinline__ int packed_head(const Write8Args& a, int role, int h) {
  if (a.sectioned) return role == kRoleQ ? h : (role == kRoleK ? a.n_q + h : a.n_q + a.n_kv + h);
  if (role != kRoleQ) return h * (a.group + 2) + a.group + (role == kRoleV);
  const int g = h / a.group;
  return g * (a.group + 2) + (h - g * a.group);
}

// One row of a head from its two chunks: bias, norm, rotation (v: the bias alone).
// The lanes of a row call it together.
template <int HD>
__device__ __forceinline__ void finish_row(const Write8Args& a, int role, int head, const uint4& xlo, const uint4& xhi,
                                           const RotUnit& ru, const float* s_w, const float* angles, int64_t token,
                                           Row& y) {
  using G = Tile<HD>;
  unpack_pairs(xlo, y.lo);
  unpack_pairs(xhi, y.hi);
  if (a.bias) {
    float2 b[4];
    const float* p = a.bias + head * HD + 8 * ru.lo;
    load_pairs(p, b);
    add_bias_pairs(y.lo, b);
    load_pairs(p + 8 * ru.dist, b);
    add_bias_pairs(y.hi, b);
  }
  if (role == kRoleV) return;
  if (a.norm) {
    const float ss = pair_head_sum<G::CPH>(chunk_partial_sq(y.lo), chunk_partial_sq(y.hi));
    const float r = rsqrtf(fmaf(ss, a.inv_head_dim, a.eps));
    const float2 rr = f2(r, r);
    const float* w = s_w + (role == kRoleQ ? 0 : HD) + 8 * ru.lo;
    float2 wl[4], wh[4];
    load_pairs(w, wl);
    load_pairs(w + 8 * ru.dist, wh);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y.lo[i] = __fmul2_rn(__fmul2_rn(y.lo[i], rr), wl[i]);
      y.hi[i] = __fmul2_rn(__fmul2_rn(y.hi[i], rr), wh[i]);
    }
  }
  if (a.rope_on) {
    float2 c[4], s[4];
    if (angles) {
      const float4 c0 = *reinterpret_cast<const float4*>(angles + ru.fa), c1 = *reinterpret_cast<const float4*>(angles + ru.fb);
      const float* sn = angles + G::HALF;
      const float4 s0 = *reinterpret_cast<const float4*>(sn + ru.fa), s1 = *reinterpret_cast<const float4*>(sn + ru.fb);
      c[0] = f2(c0.x, c0.y); c[1] = f2(c0.z, c0.w); c[2] = f2(c1.x, c1.y); c[3] = f2(c1.z, c1.w);
      s[0] = f2(s0.x, s0.y); s[1] = f2(s0.z, s0.w); s[2] = f2(s1.x, s1.y); s[3] = f2(s1.z, s1.w);
    } else {  // behind the table's end
      const int32_t p = a.pos[token];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int f = (i < 2 ? ru.fa : ru.fb - 4) + 2 * i;
        rope_cos_sin(p, a.rope.turns[f], f >= a.rope.half ? 1.f : a.rope.scale, &c[i].x, &s[i].x);
        rope_cos_sin(p, a.rope.turns[f + 1], f + 1 >= a.rope.half ? 1.f : a.rope.scale, &c[i].y, &s[i].y);
      }
    }
    rotate_unit(y.lo, y.hi, c, s, a.rope.adjacent != 0, 1.f);
  }
}

__device__ __forceinline__ float row_max(const Row& y, float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(fmaxf(fmaxf(m, fabsf(y.lo[i].x)), fmaxf(fabsf(y.lo[i].y), fabsf(y.hi[i].x))), fabsf(y.hi[i].y));
  return m;
}
// Infinities become NaN: they are codes of their own, and have no say in the scale.
__device__ __forceinline__ float no_inf(float x) { return fabsf(x) == INFINITY ? NAN : x; }
__device__ __forceinline__ void no_infs(Row& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.lo[i] = f2(no_inf(y.lo[i].x), no_inf(y.lo[i].y));
    y.hi[i] = f2(no_inf(y.hi[i].x), no_inf(y.hi[i].y));
  }
}
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float inv) {
  return make_uint2(to_e4m3x4(v[0].x * inv, v[0].y * inv, v[1].x * inv, v[1].y * inv),
                    to_e4m3x4(v[2].x * inv, v[2].y * inv, v[3].x * inv, v[3].y * inv));
}
__device__ __forceinline__ uint32_t scaled_codes(uint32_t codes, float f) {
  uint32_t lo, hi;
  from_e4m3x4(codes, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// Number of a token's block of the pool, or -1 where it is not stored.
__device__ __forceinline__ int block_of(const Write8Args& a, int64_t t) {
  const int pg = a.page[t], of = a.offset[t];
  if (pg < 0 || pg >= a.num_pages || of < 0 || of >= a.page_size) return -1;
  return pg * (a.page_size / a.block) + of / a.block;
}

// Whole warp: one head's k or v of the run of `len` tokens from t0 on.
template <int HD>
__device__ __forceinline__ void write_run(const Write8Args& a, int64_t t0, int len, int role, int h, const RotUnit& ru,
                                          const float* s_w, const float* s_tab, int64_t tab_first, int tab_rows) {
  using G = Tile<HD>;
  const int lane = threadIdx.x & 31, row = lane / G::PPH;
  const int head = packed_head(a, role, h);
  const uint4* src = a.packed + head * G::CPH + ru.lo;
  uint8_t* pool = role == kRoleK ? a.k_pool : a.v_pool;
  const int blk = block_of(a, t0);
  float* scale = (role == kRoleK ? a.k_scale : a.v_scale) + (int64_t)blk * a.n_kv + h;
  const float old_raw = *scale;
  // the run's lowest place in its block: what lies below is held
  int low = a.block;
  for (int i = lane; i < len; i += 32) low = min(low, a.offset[t0 + i] % a.block);
  low = __reduce_min_sync(0xffffffffu, low);

  auto load = [&](int pass, uint4& xlo, uint4& xhi) {
    const int i = pass * G::ROWS + row;
    xlo = xhi = make_uint4(0, 0, 0, 0);
    if (i < len) {
      const uint4* p = src + (t0 + i) * a.row_stride16;
      xlo = ld_stream(p);
      xhi = ld_stream(p + ru.dist);
    }
  };
  auto finish = [&](int pass, const uint4& xlo, const uint4& xhi, Row& y) {
    const int64_t t = t0 + min(pass * G::ROWS + row, len - 1);
    const int64_t at = t - tab_first;
    finish_row<HD>(a, role, head, xlo, xhi, ru, s_w, at < tab_rows ? s_tab + at * HD : nullptr, t, y);
  };
  auto store = [&](int pass, const Row& y, float inv) {
    const int i = pass * G::ROWS + row;
    if (i >= len) return;
    const int64_t slot = (int64_t)a.page[t0 + i] * a.page_size + a.offset[t0 + i];
    uint2* dst = reinterpret_cast<uint2*>(pool + (slot * a.n_kv + h) * HD) + ru.lo;
    dst[0] = codes8(y.lo, inv);
    dst[ru.dist] = codes8(y.hi, inv);
  };
  // the block's scale from the maximum, held codes moved, 1 / scale
  auto settle = [&](float top) {
    float s;
    if (low == 0) {
      s = fmaxf(__fdiv_rn(top, kE4m3Max), kScaleLeast);
      if (lane == 0) *scale = s;
    } else {
      const float old = clamp_scale(old_raw);
      const uint32_t t = __float_as_uint(top), m = __float_as_uint(kE4m3Max * old);
      const int k = max(0, (int)(t >> 23) - (int)(m >> 23) + ((t & 0x7fffffu) > (m & 0x7fffffu) ? 1 : 0));
      s = __uint_as_float(__float_as_uint(old) + ((uint32_t)k << 23));
      if (k > 0) {
        const float f = k > 30 ? 0.f : __uint_as_float((uint32_t)(127 - k) << 23);
        for (int i = lane; i < low * (HD / 16); i += 32) {
          uint4* p = reinterpret_cast<uint4*>(pool + (((int64_t)blk * a.block + i / (HD / 16)) * a.n_kv + h) * HD) + i % (HD / 16);
          const uint4 c = *p;
          *p = make_uint4(scaled_codes(c.x, f), scaled_codes(c.y, f), scaled_codes(c.z, f), scaled_codes(c.w, f));
        }
      }
      if (lane == 0 && s != old_raw) *scale = s;
    }
    return __frcp_rn(s);
  };

  const int passes = (len + G::ROWS - 1) / G::ROWS;
  if (passes <= kHold) {
    uint4 xlo[kHold], xhi[kHold];
    Row y[kHold];
#pragma unroll
    for (int p = 0; p < kHold; ++p)
      if (p < passes) load(p, xlo[p], xhi[p]);
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < kHold; ++p)
      if (p < passes) {
        finish(p, xlo[p], xhi[p], y[p]);
        if (p * G::ROWS + row < len) top = row_max(y[p], top);
      }
    top = warp_max(top);
    if (top == INFINITY) {
      top = 0.f;
#pragma unroll
      for (int p = 0; p < kHold; ++p)
        if (p < passes) {
          no_infs(y[p]);
          if (p * G::ROWS + row < len) top = row_max(y[p], top);
        }
      top = warp_max(top);
    }
    const float inv = settle(top);
#pragma unroll
    for (int p = 0; p < kHold; ++p)
      if (p < passes) store(p, y[p], inv);
    return;
  }
  float top = 0.f;
  for (int p = 0; p < passes; ++p) {
    uint4 xlo, xhi;
    Row y;
    load(p, xlo, xhi);
    finish(p, xlo, xhi, y);
    no_infs(y);
    if (p * G::ROWS + row < len) top = row_max(y, top);
  }
  const float inv = settle(warp_max(top));
  for (int p = 0; p < passes; ++p) {
    uint4 xlo, xhi;
    Row y;
    load(p, xlo, xhi);
    finish(p, xlo, xhi, y);
    no_infs(y);
    store(p, y, inv);
  }
}

}  // namespace

template <int HD>
__global__ void __launch_bounds__(32 * kWarps, 2) qkvp_pool_write8_kernel(const Write8Args a) {
  using G = Tile<HD>;
  extern __shared__ __align__(16) unsigned char smem[];
  float* s_tab = reinterpret_cast<float*>(smem);  // [tab_rows][cos HALF, sin HALF]
  __shared__ float s_w[2 * HD];
  __shared__ int s_start[32], s_len[32], s_runs, s_end;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int ntok = (int)min((int64_t)a.tile, a.T - t0);

  if (warp == 0) {  // the runs that begin in the tile (tile <= 32)
    const int blk = lane < ntok ? block_of(a, t0 + lane) : -1;
    int before = __shfl_up_sync(0xffffffffu, blk, 1);
    if (lane == 0) before = t0 > 0 ? block_of(a, t0 - 1) : -1;
    const bool begins = blk >= 0 && blk != before;
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    // tokens where a run cannot go on: a start, a token that is not stored, the tile's end
    const uint32_t stops = starts | __ballot_sync(0xffffffffu, blk < 0);
    int end = ntok;
    if (begins) {
      const uint32_t later = lane < 31 ? stops >> (lane + 1) : 0u;
      const int stop = later ? lane + __ffs(later) : 32;
      const int r = __popc(starts & ((1u << lane) - 1u));
      s_start[r] = lane;
      s_len[r] = min(stop, ntok) - lane;
    }
    // the last run may go on behind the tile
    const int last_blk = __shfl_sync(0xffffffffu, blk, ntok - 1);
    const int last_start = starts ? 31 - __clz(starts) : -1;
    const uint32_t within = ntok < 32 ? (1u << ntok) - 1u : 0xffffffffu;
    if (last_start >= 0 && !(stops & within & ~((2u << last_start) - 1u))) {
      for (int64_t at = t0 + ntok; at < a.T;) {
        const bool same = at + lane < a.T && block_of(a, at + lane) == last_blk;
        const uint32_t no = ~__ballot_sync(0xffffffffu, same);
        const int n = no ? __ffs(no) - 1 : 32;
        end += n;
        at += n;
        if (n < 32) break;
      }
      if (lane == 0) s_len[__popc(starts) - 1] += end - ntok;
    }
    if (lane == 0) {
      s_runs = __popc(starts);
      s_end = end;
    }
    if (a.dev_status && blockIdx.y == 0 && lane < ntok && blk < 0) {
      const int pg = a.page[t0 + lane], of = a.offset[t0 + lane];
      const int bad = (pg < 0 || pg >= a.num_pages ? QKVP_DEV_BAD_PAGE : 0) | (of < 0 || of >= a.page_size ? QKVP_DEV_BAD_OFFSET : 0);
      atomicOr(a.dev_status, bad);
    }
  }
  if (a.norm)
    for (int i = threadIdx.x; i < 2 * HD; i += 32 * kWarps) s_w[i] = i < HD ? a.w_q[i] : a.w_k[i - HD];
  __syncthreads();
  const int tab_rows = min(s_end, a.tab_rows);
  if (a.rope_on) {
    for (int i = threadIdx.x; i < tab_rows * G::HALF; i += 32 * kWarps) {
      const int tl = i / G::HALF, f = i % G::HALF;
      float c, s;
      rope_cos_sin(a.pos[t0 + tl], a.rope.turns[f], f >= a.rope.half ? 1.f : a.rope.scale, &c, &s);
      s_tab[tl * HD + f] = c;
      s_tab[tl * HD + G::HALF + f] = s;
    }
    __syncthreads();
  }

  const RotUnit ru = a.rope_on ? rot_unit<G::CPH>(lane % G::PPH, a.rope) : RotUnit{lane % G::PPH, G::PPH, 0, 4};
  const int kv_units = s_runs * 2 * a.n_kv;
  const int q_rows = ntok * a.n_q, per = G::ROWS * kQueryRows;
  const int units = kv_units + (q_rows + per - 1) / per;
  for (int u = warp + kWarps * blockIdx.y; u < units; u += kWarps * gridDim.y) {
    if (u < kv_units) {
      const int r = u / (2 * a.n_kv), x = u - r * 2 * a.n_kv;
      write_run<HD>(a, t0 + s_start[r], s_len[r], (x & 1) ? kRoleV : kRoleK, x >> 1, ru, s_w, s_tab, t0, tab_rows);
      continue;
    }
    const int row0 = (u - kv_units) * per + lane / G::PPH;
    uint4 xlo[kQueryRows], xhi[kQueryRows];
    int tok[kQueryRows], h[kQueryRows];
#pragma unroll
    for (int i = 0; i < kQueryRows; ++i) {
      const int row = min(row0 + i * G::ROWS, q_rows - 1);
      tok[i] = row / a.n_q;
      h[i] = row - tok[i] * a.n_q;
      const uint4* p = a.packed + (t0 + tok[i]) * a.row_stride16 + packed_head(a, kRoleQ, h[i]) * G::CPH + ru.lo;
      xlo[i] = ld_stream(p);
      xhi[i] = ld_stream(p + ru.dist);
    }
#pragma unroll
    for (int i = 0; i < kQueryRows; ++i) {
      Row y;
      finish_row<HD>(a, kRoleQ, packed_head(a, kRoleQ, h[i]), xlo[i], xhi[i], ru, s_w, s_tab + tok[i] * HD, t0 + tok[i], y);
      if (row0 + i * G::ROWS < q_rows) {
        uint4* dst = a.q + ((t0 + tok[i]) * a.n_q + h[i]) * G::CPH + ru.lo;
        st_keep(dst, pack_pairs(y.lo));
        st_keep(dst + ru.dist, pack_pairs(y.hi));
      }
    }
  }
}

const void* pool_write8_kernel(int head_dim) {
  return head_dim == 64 ? reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<64>)
                        : reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<128>);
}
int pool_write8_threads() { return 32 * kWarps; }

}  // namespace qkvp
