// Attention of one new token per sequence over the paged key/value pool (the
// pool that qkv_prologue_pool_write fills), split over the keys.
//
// A key's 4 D bytes (k and v of one head) meet 4 D G flops, G = n_q / n_kv query
// heads of the group: with G of 4 to 16 that is far below what the tensor cores
// could do, so the kernel is bound by reading the pool once, and its work is to
// keep enough of it in flight. Every warp is a worker of its own: it streams
// tiles of 16 or 32 keys of one key/value head through its own ring of shared memory
// (16-byte asynchronous copies, no barrier with other warps), with
//     S = Q K^T,  P = 2^(c S - m),  O += P V
// on m16n8k16 matrix instructions, the group's heads being the rows (rows past
// the group are zero). Running maxima and sums are fp32; P is rounded to bf16 as
// an operand.
//
// Split. The tiles of all sequences, one after the other, are cut into `ranges`
// equal parts, whatever the lengths are; a warp takes one head's tiles of one
// part, and neighbouring warps take neighbouring heads of the same part, so that
// the warps of an SM read whole rows of the pool (n_kv D values) between them.
// Lengths are read on the device: nothing has to be planned on the host, and a
// captured call follows lengths that grow. A sequence that lies in several parts
// leaves a partial result (m, l, O) in each; qkvp_attention_join_kernel adds
// them, and the shared prefix's, in a fixed order.
//
// Measured: 131072 keys, 32 over 8 heads of 128: 88 us, 0.89 of the copy rate (the first
// kernel 0.94; the join is a chain of dependent reads); 256 sequences of up to 4096 keys, 64
// over 8 heads of 64: 187 us, 0.93.
#include "attention.cuh"

namespace qkvp {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;

// Keys per tile and tiles in flight per warp: 8 KiB a tile, 192 KiB an SM.
template <int HD>
struct DecShape {
  static constexpr int kKeys = dec_tile_keys(HD);
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = 2 * kKeys * HD * 2;  // k rows, then v rows
  static constexpr int kWarpBytes = kStages * kTileBytes;
};

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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

}  // namespace

template <int HD>
__global__ void __launch_bounds__(kDecThreads, 1) qkvp_attention_decode_kernel(const AttnDecodeArgs a) {
  using SH = DecShape<HD>;
  constexpr int ST = SH::kStages, KT = SH::kKeys, NT = KT / 8;
  constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks per row, rows per copy instruction
  constexpr uint32_t kAll = KT == 32 ? 0xffffffffu : (1u << KT) - 1u;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint32_t s_in[kDecWarps][ST];  // bit i: key i of the stage's tile is attended
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_addr(smem_raw) + warp * SH::kWarpBytes;
  const float c = a.scale_log2;
  // Behind the prefix kernel this one begins at once: it reads nothing of that
  // kernel's, which itself waited for everything before it. It waits at its end, so
  // that the joining kernel, which waits for this one, has both.
  if (!a.prefix_chunks) griddep_wait();
  griddep_launch_dependents();

  const int64_t total = dec_total(a, lane);
  const int64_t quota = dec_quota(a, total);
  const int heads = a.n_kv * a.head_blocks;
  const int items = a.ranges * heads;
  for (int w = blockIdx.x * kDecWarps + warp; w < items; w += gridDim.x * kDecWarps) {
    const int range = w / heads;
    const int64_t t0 = range * quota;
    if (t0 >= total) break;
    const int n_tiles = (int)min(quota, total - t0);
    const int hv = w % heads, kvh = hv / a.head_blocks, hb = hv % a.head_blocks;
    const int head0 = kvh * a.group + hb * 16, n_heads = min(16, a.group - hb * 16);

    // where the range begins
    DecCursor cu{0, 0, 0};
    {
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
    }

    // Loads run ST - 1 tiles ahead of the arithmetic, and the page lookup of a
    // tile one step ahead of its loads.
    DecCursor ld = cu;
    uint32_t ld_keys = (uint32_t)(a.joint_len + dec_own(a, ld.b));
    int slot = -1;
    auto look_up = [&]() {
      if (lane < KT) slot = dec_slot(a, ld.b, ld_keys, (uint32_t)(ld.tile * KT + lane));
    };
    auto advance = [&]() {
      if (++ld.tile < ld.tiles) return;
      ld.settle(a, lane);
      ld_keys = (uint32_t)(a.joint_len + dec_own(a, ld.b));
    };
    const int ch = lane % CH, row_ch = a.n_kv * CH;
    const uint4* k_src = a.k_pool + kvh * CH + ch;
    const uint4* v_src = a.v_pool + kvh * CH + ch;
    auto issue = [&](uint32_t st) {
      const uint32_t in = __ballot_sync(0xffffffffu, lane < KT && slot >= 0);
      if (lane == 0) s_in[warp][st] = in;
      const uint32_t dst = ring + st * SH::kTileBytes;
#pragma unroll
      for (int i = 0; i < KT / RPI; ++i) {
        const int r = i * RPI + lane / CH;
        const int row = __shfl_sync(0xffffffffu, slot, r);
        const int64_t off = (int64_t)max(row, 0) * row_ch;
        const uint32_t to = dst + r * (HD * 2) + ((ch ^ (r & 7)) << 4);
        cp_async16(to, k_src + off, row >= 0);
        cp_async16(to + KT * HD * 2, v_src + off, row >= 0);
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

    uint32_t qf[HD / 16][4];
    float o[HD / 8][4], m[2], l[2];  // m in powers of two (the scores times scale log2(e))
    auto begin = [&]() {             // a sequence's first tile here
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = (lane >> 2) + 8 * (x & 1), d = 16 * ks + 8 * (x >> 1) + 2 * (lane & 3);
          qf[ks][x] =
              r < n_heads ? *reinterpret_cast<const uint32_t*>(a.q + ((int64_t)cu.b * a.n_q + head0 + r) * HD + d) : 0u;
        }
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    };
    bool first = cu.tile == 0;  // of the sequence: else the segment continues one of the range before
    auto end = [&]() {          // its last tile here: the partial result
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = (lane >> 2) + 8 * x;
        if (r < n_heads) {
          const int64_t row = (int64_t)(first ? cu.b : a.batch + range) * a.n_q + head0 + r;
          if ((lane & 3) == 0) a.part_ml[row] = make_float2(m[x], l[x]);
          float2* dst = reinterpret_cast<float2*>(a.part_o + row * HD) + (lane & 3);
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) dst[4 * i] = make_float2(o[i][2 * x], o[i][2 * x + 1]);
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
      const uint32_t kt = ring + st * SH::kTileBytes, vt = kt + KT * HD * 2;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      {
        const int key = ((lane >> 4) << 3) + (lane & 7), hi = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm4(kt + (8 * n + key) * (HD * 2) + (((2 * ks + hi) ^ (key & 7)) << 4), b);
            mma16816(s[n], qf[ks], b[0], b[1]);
            mma16816(s[n + 1], qf[ks], b[2], b[3]);
          }
      }
      const uint32_t in = s_in[warp][st];
      if (in != kAll) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (!((in >> (8 * n + 2 * (lane & 3) + (x & 1))) & 1)) s[n][x] = -INFINITY;
      }
      // A row's reference m only moves where a score passes it by more than 8 powers of
      // two (see the prompt kernel); until then no lane has to know the others' maxima.
      float top[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(s[0][2 * x], s[0][2 * x + 1]);
#pragma unroll
        for (int n = 1; n < NT; ++n) top[x] = max3(top[x], s[n][2 * x], s[n][2 * x + 1]);
      }
      if (__any_sync(0xffffffffu, fmaf(top[0], c, -m[0]) > 8.f || fmaf(top[1], c, -m[1]) > 8.f)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = top[x] * c;
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          const float m_new = fmaxf(m[x], v);
          const float f = m_new == m[x] ? 1.f : ex2(m[x] - m_new);
          m[x] = m_new;
          l[x] *= f;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            o[i][2 * x] *= f;
            o[i][2 * x + 1] *= f;
          }
        }
      }
      uint32_t pf[NT / 2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float off = m[x] == -INFINITY ? 0.f : -m[x];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float p0 = ex2(fmaf(s[n][2 * x], c, off)), p1 = ex2(fmaf(s[n][2 * x + 1], c, off));
          l[x] += p0 + p1;
          pf[n >> 1][2 * (n & 1) + x] = pack2(p0, p1);
        }
      }
      {
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), hi = lane >> 4;
#pragma unroll
        for (int k2 = 0; k2 < NT / 2; ++k2)
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            uint32_t b[4];
            ldsm4t(vt + (16 * k2 + key) * (HD * 2) + (((2 * i + hi) ^ (key & 7)) << 4), b);
            mma16816(o[2 * i], pf[k2], b[0], b[1]);
            mma16816(o[2 * i + 1], pf[k2], b[2], b[3]);
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
  if (a.prefix_chunks) griddep_wait();
}

// Joins the partial results of each (sequence, head): its own in the ranges it
// lies in and the shared prefix's key ranges, in that order. kJoinWarps warps per
// CTA, `wph` of them per head. A chain of dependent reads (lengths, maxima and
// sums, results), so each is made by as many lanes at once as there are.
template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) qkvp_attention_join_kernel(const AttnDecodeArgs a) {
  constexpr int V = HD / 32;             // values per lane
  constexpr int kCap = kJoinParts / kJoinWarps;  // factors in shared memory per warp
  __shared__ float s_f[kJoinParts], s_top[kJoinWarps], s_sum[kJoinWarps], s_o[kJoinWarps][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wph = a.wph, per = kJoinWarps / wph;  // heads per CTA
  const int groups = (a.n_q + per - 1) / per;
  const int b = (int)(blockIdx.x / groups), grp = warp / wph, sub = warp % wph;
  const int head = (int)(blockIdx.x % groups) * per + grp, tid = 32 * sub + lane;
  griddep_wait();
  griddep_launch_dependents();
  const int2 plan = a.plan[b];  // means nothing where the sequence has no tile
  const int length = a.lengths[b];
  if (threadIdx.x == 0 && blockIdx.x % groups == 0 && a.dev_status &&
      (length < 0 || length > a.max_pages * a.page_size))
    atomicOr(a.dev_status, kDevBadLength);
  const int own = dec_tiles(a, b) ? plan.y - plan.x + 1 : 0, parts = own + a.prefix_chunks;
  const bool on = head < a.n_q;
  // row of partial result i in part_o / part_ml: [batch] first pieces, [ranges] later ones, [prefix chunks][batch]
  auto row_of = [&](int i) -> int64_t {
    const int64_t r = i == 0 && own ? (int64_t)b
                      : i < own     ? (int64_t)a.batch + plan.x + i
                                    : (int64_t)a.batch + a.ranges + (int64_t)(i - own) * a.batch + b;
    return r * a.n_q + head;
  };
  float top = -INFINITY, sum = 0.f, o[V] = {};
#pragma unroll 4
  for (int i = on ? tid : parts; i < parts; i += 32 * wph) top = fmaxf(top, a.part_ml[row_of(i)].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  for (int x = 0; x < wph; ++x) top = fmaxf(top, s_top[grp * wph + x]);
  const float off = top == -INFINITY ? 0.f : top;
  float* f = s_f + grp * wph * kCap;
  for (int i0 = 0; i0 < parts; i0 += kCap * wph) {  // as many parts as factors fit
    const int n = min(kCap * wph, parts - i0);
    if (i0) __syncthreads();
    for (int i = on ? tid : n; i < n; i += 32 * wph) {
      const float2 v = a.part_ml[row_of(i0 + i)];
      f[i] = ex2(v.x - off);
      sum += f[i] * v.y;
    }
    __syncthreads();
    for (int i = on ? sub : n; i < n; i += 8 * wph) {
      float v[8][V];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int ik = min(i + k * wph, n - 1);
        const float* src = a.part_o + row_of(i0 + ik) * HD + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = src[e];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float fk = i + k * wph < n ? f[i + k * wph] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fk != 0.f ? fmaf(fk, v[k][e], o[e]) : o[e];
      }
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (wph > 1) {
    if (lane == 0) s_sum[warp] = sum;
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][V * lane + e] = o[e];
    __syncthreads();
    if (sub == 0)
      for (int x = 1; x < wph; ++x) {
        sum += s_sum[warp + x];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += s_o[warp + x][V * lane + e];
      }
  }
  if (!on || sub != 0) return;
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((int64_t)b * a.n_q + head) * HD) + V / 2 * lane;
#pragma unroll
  for (int e = 0; e < V / 2; ++e) dst[e] = pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)b * a.n_q + head] = (top + log2f(sum)) * 0.6931471805599453f;
}

const void* attention_decode_kernel(int head_dim) {
  return head_dim == 64 ? reinterpret_cast<const void*>(&qkvp_attention_decode_kernel<64>)
                        : reinterpret_cast<const void*>(&qkvp_attention_decode_kernel<128>);
}
const void* attention_join_kernel(int head_dim) {
  return head_dim == 64 ? reinterpret_cast<const void*>(&qkvp_attention_join_kernel<64>)
                        : reinterpret_cast<const void*>(&qkvp_attention_join_kernel<128>);
}
int attention_decode_smem_bytes(int head_dim) {
  return kDecWarps * (head_dim == 64 ? DecShape<64>::kWarpBytes : DecShape<128>::kWarpBytes);
}
int attention_decode_threads() { return kDecThreads; }
int attention_decode_warps() { return kDecWarps; }

}  // namespace qkvp
