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
// Work. A CTA, or several along y that divide its units, takes `tile` tokens. The tokens of one
// block that follow each other are a run; the CTAs whose tile has a run's first token do the
// whole run, k or v of a head in one warp (of short runs, of a few heads). A row of a head is
// CPH / 2 lanes, two chunks of 8 values each (the units of rot_unit), so a warp holds 4 or 8
// rows at once: of a run that many tokens of one head, of a shorter run several heads too (a
// decode step's runs are single tokens). A warp works in steps of four times that, 4 KiB of
// rows, of query heads or of one head's k or v of a run. It has two buffers in shared memory
// and copies the next step's rows (asynchronously) while it works on one: what is in flight
// takes no registers, and a run of one step is gone over twice, for amax and for the codes,
// without being read again. A longer run is read twice, the second time from L2.
//
// cos and sin of the tile's tokens are computed once per CTA into shared memory, for all
// its heads (query heads of one token follow each other, so a lane keeps a token's in
// registers); tokens of a run beyond the table's end get theirs computed by the lanes that
// use them.
//
// Bound by instructions: 16384 tokens, 32 over 8 heads of 128, blocks of 16, take 83 to 86 us,
// 4.4 TB/s or 0.64 of a plain copy's rate, with 54 % of the issue slots used by the 16 warps that
// 119 to 124 registers leave room for. 4001 tokens behind 100 held ones (64 over 8 heads of 64, blocks
// of 8, bias): 30 us in one wave of CTAs. In longer blocks what a warp's run takes: 4096 tokens of
// the first heads 27 us in blocks of 16, 46 of 64, 218 of 256. 256 single tokens (128 over 16 heads of 64): 8 us,
// the chain of reads of one CTA.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "pipeline.cuh"
#include "qkv_prologue.h"

namespace qkvp {
namespace {

constexpr int kWarps = 8;
constexpr int kPasses = 4;         // times the rows that a warp holds: a step
constexpr int kStepBytes = 4096;

// A row's two chunks as they are stored, and widened.
struct Raw {
  uint4 lo, hi;
};
struct Row {
  float2 lo[4], hi[4];
};

template <int HD>
struct Tile {
  static constexpr int CPH = HD / 8, PPH = CPH / 2;
  static constexpr int ROWS = 32 / PPH;  // rows of a head that a warp holds at once
};

__device__ __forceinline__ uint32_t quotient(uint32_t n, const SmallDiv& d) { return d.magic ? small_div(n, d.magic) : n; }

// Position of a head in the packed row.
__device__ __forceinline__ int packed_head(const Write8Args& a, int role, int h) {
  if (a.sectioned) return role == kRoleQ ? h : (role == kRoleK ? a.n_q + h : a.n_q + a.n_kv + h);
  if (role != kRoleQ) return h * (a.group + 2) + a.group + (role == kRoleV);
  return h + 2 * (int)quotient((uint32_t)h, a.by_group);
}

// Four floats from shared memory where they are used: the compiler would hold weights
// and angles in registers across loops, and spill.
__device__ __forceinline__ float4 read4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_addr(p)));
  return v;
}

__device__ __forceinline__ void add_bias4(const float* p, float2 (&y)[4]) {
  float2 b[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("ld.global.nc.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(b[2 * i].x), "=f"(b[2 * i].y), "=f"(b[2 * i + 1].x), "=f"(b[2 * i + 1].y)
                 : "l"(p + 4 * i));
  add_bias_pairs(y, b);
}
template <int HD, bool BIAS>
__device__ __forceinline__ void widen(const Write8Args& a, int head, const Raw& x, const RotUnit& ru, Row& y) {
  unpack_pairs(x.lo, y.lo);
  unpack_pairs(x.hi, y.hi);
  if (BIAS) {
    const float* p = a.bias + head * HD + 8 * ru.lo;
    add_bias4(p, y.lo);
    add_bias4(p + 8 * ru.dist, y.hi);
  }
}
// The norm's weights of a lane's values.
struct Weights {
  float2 lo[4], hi[4];
};
__device__ __forceinline__ void read_weights(const float* weights, const RotUnit& ru, Weights& w) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 l = read4(weights + 8 * ru.lo + 4 * i), h = read4(weights + 8 * (ru.lo + ru.dist) + 4 * i);
    w.lo[2 * i] = f2(l.x, l.y);
    w.lo[2 * i + 1] = f2(l.z, l.w);
    w.hi[2 * i] = f2(h.x, h.y);
    w.hi[2 * i + 1] = f2(h.z, h.w);
  }
}
// The norm of a row (its lanes together).
template <int HD>
__device__ __forceinline__ void norm_row(const Write8Args& a, const Weights& w, Row& y) {
  const float ss = pair_head_sum<HD / 8>(chunk_partial_sq(y.lo), chunk_partial_sq(y.hi));
  const float r = rsqrtf(fmaf(ss, a.inv_head_dim, a.eps));
  const float2 rr = f2(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y.lo[i] = __fmul2_rn(__fmul2_rn(y.lo[i], rr), w.lo[i]);
    y.hi[i] = __fmul2_rn(__fmul2_rn(y.hi[i], rr), w.hi[i]);
  }
}

// cos, sin and -sin of a lane's values.
struct Angles {
  float2 c[4], s[4], n[4];
  __device__ __forceinline__ void negate() {
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = f2(-s[i].x, -s[i].y);
  }
};
// rotate_unit with the negatives at hand.
template <int ROPE>
__device__ __forceinline__ void turn_row(const Write8Args& a, const RotUnit& ru, const Angles& g, Row& y) {
  if (ROPE == kRopeAdjacent) {
    rotate_unit(y.lo, y.hi, g.c, g.s, a.rope, ru, 1.f);
    return;
  }
  if (!ru.first_turns(a.rope)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __ffma2_rn(y.lo[i], g.c[i], __fmul2_rn(y.hi[i], g.n[i]));
    y.hi[i] = __ffma2_rn(y.hi[i], g.c[i], __fmul2_rn(y.lo[i], g.s[i]));
    y.lo[i] = p;
  }
}
template <int HD>
__device__ __forceinline__ void read_angles(const float* row, const RotUnit& ru, Angles& g) {
  const float* sn = row + HD / 2;
  const float4 c0 = read4(row + ru.fa), c1 = read4(row + ru.fb), s0 = read4(sn + ru.fa), s1 = read4(sn + ru.fb);
  g.c[0] = f2(c0.x, c0.y); g.c[1] = f2(c0.z, c0.w); g.c[2] = f2(c1.x, c1.y); g.c[3] = f2(c1.z, c1.w);
  g.s[0] = f2(s0.x, s0.y); g.s[1] = f2(s0.z, s0.w); g.s[2] = f2(s1.x, s1.y); g.s[3] = f2(s1.z, s1.w);
  g.negate();
}
// The same of a token behind the table's end.
__device__ __forceinline__ void make_angles(const Write8Args& a, int64_t token, const RotUnit& ru, Angles& g) {
  const int32_t p = a.pos[token];
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int f = (i < 2 ? ru.fa : ru.fb - 4) + 2 * i;
    float2 c, s;
    rope_cos_sin(p, a.rope.turns[f], a.rope.scale, &c.x, &s.x);
    rope_cos_sin(p, a.rope.turns[f + 1], a.rope.scale, &c.y, &s.y);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j == i) {
        g.c[j] = c;
        g.s[j] = s;
      }
  }
  g.negate();
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
// A block's scale s and 1 / s, the nearest float32. x / s to the nearest float32 from them: y =
// x (1 / s) lies within two of its last places; y s - x is exact in one operation, and y less
// that times 1 / s is the quotient but for its rounding (Markstein, 1990). y alone puts one
// code in 2000 of bf16 values on the other side of a near tie.
struct Scale {
  float s, inv;
};
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], const Scale& sc) {
  float2 x[4];
  const float2 s = f2(sc.s, sc.s), neg = f2(-sc.inv, -sc.inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 nx = f2(-v[i].x, -v[i].y), y = __fmul2_rn(nx, neg);  // (of -x: a zero keeps its sign)
    x[i] = __ffma2_rn(__ffma2_rn(y, s, nx), neg, y);
  }
  return make_uint2(to_e4m3x4(x[0].x, x[0].y, x[1].x, x[1].y), to_e4m3x4(x[2].x, x[2].y, x[3].x, x[3].y));
}
__device__ __forceinline__ uint32_t scaled_codes(uint32_t codes, float f) {
  uint32_t lo, hi;
  from_e4m3x4(codes, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// max(m, |x|) over a row of bf16 (a NaN is passed over, as fmaxf does).
__device__ __forceinline__ float raw_max(const Raw& x, float m) {
  const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
  __nv_bfloat162 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
#pragma unroll
  for (int n = 4; n; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = __hmax2(t[i], t[i + n]);
  return fmaxf(m, fmaxf(__low2float(t[0]), __high2float(t[0])));
}

// Number of a token's block of the pool, or -1 where it is not stored.
__device__ __forceinline__ int block_of(const Write8Args& a, int pg, int of) {
  if (pg < 0 || pg >= a.num_pages || of < 0 || of >= a.page_size) return -1;
  const int slot = pg * a.page_size + of;  // (a page is whole blocks)
  return a.block_shift >= 0 ? slot >> a.block_shift : slot / a.block;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ Raw read_raw(uint32_t at, int dist) {
  Raw x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.lo.x), "=r"(x.lo.y), "=r"(x.lo.z), "=r"(x.lo.w) : "r"(at));
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.hi.x), "=r"(x.hi.y), "=r"(x.hi.z), "=r"(x.hi.w)
               : "r"(at + 16 * dist));
  return x;
}

// k or v of a run, of the heads h0 .. that a warp's rows have room for; 1 << ts rows are
// tokens of one head.
struct RunUnit {
  int64_t t0;  // first token
  int len, blk, low;
  int page0;   // its page's first slot
  int ts;
  int role, h0;
  __device__ __forceinline__ int passes() const { return (len + (1 << ts) - 1) >> ts; }
  __device__ __forceinline__ int chunks() const { return (passes() + kPasses - 1) / kPasses; }
};

// Whole warp: the unit's block scale from amax (over each head's lanes), held codes
// moved where it grows.
template <int HD>
__device__ __forceinline__ Scale settle_scale(const Write8Args& a, const RunUnit& u, int h, bool mine, float top) {
  using G = Tile<HD>;
  float* scale = (u.role == kRoleK ? a.k_scale : a.v_scale) + (int64_t)u.blk * a.n_kv + h;
  const int part = (threadIdx.x & 31) & ((G::PPH << u.ts) - 1);  // lane within the head
  float s;
  if (u.low == 0) {
    s = fmaxf(__fdiv_rn(top, kE4m3Max), kScaleLeast);
    if (part == 0 && mine) *scale = s;
  } else {
    const float old_raw = *scale, old = clamp_scale(old_raw);
    const uint32_t t = __float_as_uint(top), m = __float_as_uint(kE4m3Max * old);
    const int k = max(0, (int)(t >> 23) - (int)(m >> 23) + ((t & 0x7fffffu) > (m & 0x7fffffu) ? 1 : 0));
    s = __uint_as_float(__float_as_uint(old) + ((uint32_t)k << 23));
    if (k > 0 && mine) {
      const float f = k > 30 ? 0.f : __uint_as_float((uint32_t)(127 - k) << 23);
      uint4* first = reinterpret_cast<uint4*>((u.role == kRoleK ? a.k_pool : a.v_pool) +
                                              ((int64_t)u.blk * a.block * a.n_kv + h) * HD);
#pragma unroll 2
      for (int i = part; i < u.low * (HD / 16); i += G::PPH << u.ts) {
        uint4* p = first + (int64_t)(i / (HD / 16)) * a.n_kv * (HD / 16) + i % (HD / 16);
        const uint4 c = *p;
        *p = make_uint4(scaled_codes(c.x, f), scaled_codes(c.y, f), scaled_codes(c.z, f), scaled_codes(c.w, f));
      }
    }
    __syncwarp();  // (all lanes of a head have its old scale)
    if (part == 0 && mine && s != old_raw) *scale = s;
  }
  return Scale{s, __frcp_rn(s)};
}

// What a warp keeps of a run between the steps that it takes.
struct RunState {
  float top;
  Scale scale;
  bool inf;
};

// Whole warp: a step of a unit of k or v: rows in buf. A run of one chunk is done in its
// one step; else the first chunks() steps find amax, and as many more write.
template <int HD, int ROPE, bool NORM, bool BIAS>
__device__ __forceinline__ void run_step(const Write8Args& a, const RunUnit& u, int step, uint32_t buf, const RotUnit& ru,
                                         const float* s_w, const float* s_tab, int64_t tab_first, int tab_rows,
                                         RunState& st) {
  using G = Tile<HD>;
  const int lane = threadIdx.x & 31, row = lane / G::PPH, tok = row & ((1 << u.ts) - 1);
  const int h = min(u.h0 + (row >> u.ts), a.n_kv - 1);
  const bool mine = u.h0 + (row >> u.ts) < a.n_kv, key = u.role == kRoleK;
  const int head = packed_head(a, u.role, h), chunks = u.chunks();
  const int chunk = step < chunks ? step : step - chunks, pass0 = chunk * kPasses, n = min(kPasses, u.passes() - pass0);
  buf += (uint32_t)(row * (HD * 2) + 16 * ru.lo);
  const bool plain = !key && !BIAS;  // bf16 as it is
  const int i0 = (pass0 << u.ts) + tok;
  auto row_at = [&](int p, Row& y) {  // the values of this lane's row of the chunk's pass
    widen<HD, BIAS>(a, head, read_raw(buf + p * 1024, ru.dist), ru, y);
    if (key) {
      if (NORM) {
        Weights w;
        read_weights(s_w + HD, ru, w);
        norm_row<HD>(a, w, y);
      }
      if (ROPE) {
        const int at = (int)(u.t0 - tab_first) + min(i0 + (p << u.ts), u.len - 1);
        Angles g;
        if (at < tab_rows) read_angles<HD>(s_tab + at * HD, ru, g);
        else make_angles(a, tab_first + at, ru, g);
        turn_row<ROPE>(a, ru, g, y);
      }
    }
    if (st.inf || chunks > 1) no_infs(y);
  };
  if (step < chunks) {
    if (step == 0) {
      st.top = 0.f;
      st.inf = false;
    }
    for (;;) {
      if (plain && !st.inf && chunks == 1) {
#pragma unroll 2
        for (int p = 0; p < n; ++p)
          if (i0 + (p << u.ts) < u.len) st.top = raw_max(read_raw(buf + p * 1024, ru.dist), st.top);
      } else {
#pragma unroll 1
        for (int p = 0; p < n; ++p) {
          Row y;
          row_at(p, y);
          if (i0 + (p << u.ts) < u.len) st.top = row_max(y, st.top);
        }
      }
      if (step + 1 < chunks) return;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {  // over the lanes of a head's rows
        const float x = __shfl_xor_sync(0xffffffffu, st.top, o);
        if (o < G::PPH << u.ts) st.top = fmaxf(st.top, x);
      }
      if (!__any_sync(0xffffffffu, st.top == INFINITY)) break;
      st.inf = true;  // once more without them
      st.top = 0.f;
    }
    st.scale = settle_scale<HD>(a, u, h, mine, st.top);
    if (chunks > 1) return;
  }
  const int32_t* offset = a.offset + u.t0;
  uint2* pool = reinterpret_cast<uint2*>(key ? a.k_pool : a.v_pool) + h * (HD / 8) + ru.lo;
#pragma unroll 1
  for (int p = 0; p < n; ++p) {
    Row y;
    const int i = i0 + (p << u.ts), of = offset[min(i, u.len - 1)];
    row_at(p, y);
    if (i < u.len && mine) {
      uint2* dst = pool + (int64_t)(u.page0 + of) * (a.n_kv * (HD / 8));
      dst[0] = codes8(y.lo, st.scale);
      dst[ru.dist] = codes8(y.hi, st.scale);
    }
  }
}

// cos and sin of tokens first .. last - 1 of the tile into the table, by `threads` threads.
template <int HD>
__device__ __forceinline__ void fill_table(const Write8Args& a, float* s_tab, int64_t t0, int first, int last, int thread,
                                           int threads) {
  constexpr int HALF = HD / 2;
  for (int i = first * HALF + thread; i < last * HALF; i += threads) {
    const int tl = i / HALF, f = i % HALF;
    float c, s;
    rope_cos_sin(a.pos[t0 + tl], a.rope.turns[f], a.rope.scale, &c, &s);
    s_tab[tl * HD + f] = c;
    s_tab[tl * HD + HALF + f] = s;
  }
}

}  // namespace

template <int HD, int ROPE, bool NORM, bool BIAS>
__global__ void __launch_bounds__(32 * kWarps, 2) qkvp_pool_write8_kernel(const __grid_constant__ Write8Args a) {
  using G = Tile<HD>;
  constexpr int LOG_ROWS = G::ROWS == 8 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  // each warp's two buffers, then the table [tab_rows][cos HALF, sin HALF]
  float* s_tab = reinterpret_cast<float*>(smem + kWarps * 2 * kStepBytes);
  __shared__ __align__(16) float s_w[2 * HD];
  // the tile's runs: first token, length, block, lowest place in the block, its page's first
  // slot, log2 of the tokens side by side, units of work before it
  __shared__ int s_start[32], s_len[32], s_blk[32], s_low[32], s_page0[32], s_ts[32], s_before[33], s_runs, s_end;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int ntok = (int)min((int64_t)a.tile, a.T - t0);

  if (warp == 0) {  // the runs that begin in the tile (tile <= 32)
    int pg = -1, of = 0;
    if (lane < ntok) {
      pg = a.page[t0 + lane];
      of = a.offset[t0 + lane];
    }
    const int blk = block_of(a, pg, of);
    int before = __shfl_up_sync(0xffffffffu, blk, 1);
    if (lane == 0) before = t0 > 0 ? block_of(a, a.page[t0 - 1], a.offset[t0 - 1]) : -1;
    const bool begins = blk >= 0 && blk != before;
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    // tokens where a run cannot go on: a start, a token that is not stored, the tile's end
    const uint32_t stops = starts | __ballot_sync(0xffffffffu, blk < 0);
    const int place = pg * a.page_size + of - blk * a.block;  // in its block
    const int runs = __popc(starts), r = __popc(starts & ((1u << lane) - 1u));
    if (begins) {
      const uint32_t later = lane < 31 ? stops >> (lane + 1) : 0u;
      s_start[r] = lane;
      s_len[r] = min(later ? lane + __ffs(later) : 32, ntok) - lane;
      s_blk[r] = blk;
      s_low[r] = place;
      s_page0[r] = pg * a.page_size;
    }
    __syncwarp();
    // a token's run is the last that began up to it
    const int run = __popc(starts & (0xffffffffu >> (31 - lane))) - 1;
    if (blk >= 0 && run >= 0 && !begins && blk == s_blk[run]) atomicMin(&s_low[run], place);
    int end = ntok;
    // the last run may go on behind the tile
    const int last_start = starts ? 31 - __clz(starts) : -1;
    const uint32_t within = ntok < 32 ? (1u << ntok) - 1u : 0xffffffffu;
    if (last_start >= 0 && !(stops & within & ~((2u << last_start) - 1u))) {
      const int last_blk = __shfl_sync(0xffffffffu, blk, last_start);
      int low = a.block;
      for (int64_t at = t0 + ntok; at < a.T;) {
        const bool in = at + lane < a.T;
        const int p = in ? a.page[at + lane] : -1, o = in ? a.offset[at + lane] : 0;
        const uint32_t no = ~__ballot_sync(0xffffffffu, block_of(a, p, o) == last_blk);
        const int n = no ? __ffs(no) - 1 : 32;
        if (lane < n) low = min(low, p * a.page_size + o - last_blk * a.block);
        end += n;
        at += n;
        if (n < 32) break;
      }
      low = __reduce_min_sync(0xffffffffu, low);
      __syncwarp();  // (the minima above are in s_low)
      if (lane == 0) {
        s_len[runs - 1] += end - ntok;
        s_low[runs - 1] = min(s_low[runs - 1], low);
      }
    }
    __syncwarp();
    int units = 0;
    if (lane < runs) {
      const int ts = min(LOG_ROWS, s_len[lane] > 1 ? 32 - __clz(s_len[lane] - 1) : 0), per = G::ROWS >> ts;
      s_ts[lane] = ts;
      units = 2 * ((a.n_kv + per - 1) / per);
    }
    int upto = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    s_before[lane + 1] = upto;
    if (lane == 0) {
      s_before[0] = 0;
      s_runs = runs;
      s_end = end;
    }
    if (a.dev_status && blockIdx.y == 0 && lane < ntok && blk < 0)
      atomicOr(a.dev_status, (pg < 0 || pg >= a.num_pages ? QKVP_DEV_BAD_PAGE : 0) |
                                 (of < 0 || of >= a.page_size ? QKVP_DEV_BAD_OFFSET : 0));
  }
  if (NORM)
    for (int i = threadIdx.x; i < 2 * HD; i += 32 * kWarps) s_w[i] = i < HD ? a.w_q[i] : a.w_k[i - HD];
  if (ROPE && warp > 0) fill_table<HD>(a, s_tab, t0, 0, ntok, threadIdx.x - 32, 32 * (kWarps - 1));

  const RotUnit ru = ROPE ? rot_unit<G::CPH>(lane % G::PPH, a.rope) : RotUnit{lane % G::PPH, G::PPH, 0, 4};
  const int row = lane / G::PPH;
  // The rows of query heads in their order in q, token by token: a pass takes the warp's next
  // rows, so where they go to needs no arithmetic.
  const int q_rows = ntok * a.n_q, q_units = (q_rows + kPasses * G::ROWS - 1) / (kPasses * G::ROWS);
  const uint32_t buffers = smem_addr(smem) + warp * 2 * kStepBytes;
  const uint32_t lane_at = (uint32_t)(row * (HD * 2) + 16 * ru.lo);
  const uint4* q_src = a.packed + t0 * a.row_stride16 + ru.lo;
  uint4* q_dst = a.q + t0 * a.n_q * G::CPH + ru.lo;
  int kv_units = 0, runs = 0;  // (known behind the barrier)
  auto run_unit = [&](int u) {
    u -= q_units;
    const int r = __popc(__ballot_sync(0xffffffffu, lane < runs && s_before[lane + 1] <= u)), x = u - s_before[r];
    // k of all heads, then v: neighbouring warps have the same, and each some of both
    const int half = (s_before[r + 1] - s_before[r]) >> 1;
    return RunUnit{t0 + s_start[r], s_len[r], s_blk[r], s_low[r], s_page0[r], s_ts[r], x >= half ? (int)kRoleV : (int)kRoleK,
                   (x >= half ? x - half : x) * (G::ROWS >> s_ts[r])};
  };
  auto fetch_queries = [&](int u, uint32_t to) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int n = (u * kPasses + p) * G::ROWS + row;
      if (n < q_rows) {  // (rows that are not are never used)
        const int tok = (int)quotient((uint32_t)n, a.by_n_q), h = n - tok * a.n_q;
        const uint4* y = q_src + tok * a.row_stride16 + packed_head(a, kRoleQ, h) * G::CPH;
        copy16(to + lane_at + p * 1024, y);
        copy16(to + lane_at + p * 1024 + 16 * ru.dist, y + ru.dist);
      }
    }
  };
  auto fetch_run = [&](int u, int step, uint32_t to) {
    const RunUnit k = run_unit(u);
    const int chunks = k.chunks(), chunk = step < chunks ? step : step - chunks;
    const int h = min(k.h0 + (row >> k.ts), a.n_kv - 1), tok = row & ((1 << k.ts) - 1);
    const uint4* src = a.packed + packed_head(a, k.role, h) * G::CPH + ru.lo;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = ((chunk * kPasses + p) << k.ts);
      if (i < k.len) {
        const uint4* x = src + (k.t0 + min(i + tok, k.len - 1)) * a.row_stride16;
        copy16(to + lane_at + p * 1024, x);
        copy16(to + lane_at + p * 1024 + 16 * ru.dist, x + ru.dist);
      }
    }
  };

  const int stride = kWarps * gridDim.y;
  int u = warp + kWarps * blockIdx.y;
  uint32_t here = buffers, there = buffers + kStepBytes;
  if (u < q_units) fetch_queries(u, here);  // before the barrier: it needs nothing of the runs
  __syncthreads();
  const int tab_rows = min(s_end, a.tab_rows);
  if (ROPE && tab_rows > ntok) {
    fill_table<HD>(a, s_tab, t0, ntok, tab_rows, threadIdx.x, 32 * kWarps);
    __syncthreads();
  }
  runs = s_runs;
  kv_units = s_before[32];
  const int units = q_units + kv_units;
  if (u >= q_units && u < units) fetch_run(u, 0, here);
  asm volatile("cp.async.commit_group;" ::: "memory");
  // Behind each step's rows are the next step's on their way.
  auto fetch_next = [&](int next, int next_step) {
    if (next < q_units) fetch_queries(next, there);
    else if (next < units) fetch_run(next, next_step, there);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // (a lane reads only what it copied itself)
  };
  auto turn_over = [&]() {
    const uint32_t x = here;
    here = there;
    there = x;
  };
  {
    Weights w;
    if (NORM) read_weights(s_w, ru, w);
    Angles angles;
    int angles_of = -1;  // the token whose angles these are
    for (; u < q_units; u += stride) {
      fetch_next(u + stride, 0);
      int n = u * kPasses * G::ROWS + row;
      uint4* dst = q_dst + n * G::CPH;
      uint32_t from = here + lane_at;
#pragma unroll 1
      for (int p = 0; p < kPasses; ++p) {
        if (n - row >= q_rows) break;
        const int tok = (int)quotient((uint32_t)min(n, q_rows - 1), a.by_n_q);
        if (ROPE && tok != angles_of) {
          read_angles<HD>(s_tab + tok * HD, ru, angles);
          angles_of = tok;
        }
        Row y;
        widen<HD, BIAS>(a, BIAS ? packed_head(a, kRoleQ, min(n, q_rows - 1) - tok * a.n_q) : 0, read_raw(from, ru.dist), ru, y);
        if (NORM) norm_row<HD>(a, w, y);
        if (ROPE) turn_row<ROPE>(a, ru, angles, y);
        if (n < q_rows) {
          st_keep(dst, pack_pairs(y.lo));
          st_keep(dst + ru.dist, pack_pairs(y.hi));
        }
        n += G::ROWS;
        dst += G::ROWS * G::CPH;
        from += 1024;
      }
      turn_over();
    }
  }
  RunState st{0.f, {0.f, 0.f}, false};
  for (int step = 0; u < units;) {
    const RunUnit k = run_unit(u);
    const int chunks = k.chunks();
    const bool more = chunks > 1 && step + 1 < 2 * chunks;
    fetch_next(more ? u : u + stride, more ? step + 1 : 0);
    run_step<HD, ROPE, NORM, BIAS>(a, k, step, here, ru, s_w, s_tab, t0, tab_rows, st);
    step = more ? step + 1 : 0;
    if (!more) u += stride;
    turn_over();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int HD, bool BIAS>
const void* pool_write8_pick(int rope, bool norm) {
  if (rope == kRopeNone)
    return norm ? reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeNone, true, BIAS>)
                : reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeNone, false, BIAS>);
  if (rope == kRopeHalves)
    return norm ? reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeHalves, true, BIAS>)
                : reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeHalves, false, BIAS>);
  return norm ? reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeAdjacent, true, BIAS>)
              : reinterpret_cast<const void*>(&qkvp_pool_write8_kernel<HD, kRopeAdjacent, false, BIAS>);
}

}  // namespace qkvp
