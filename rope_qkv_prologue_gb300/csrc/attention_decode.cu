// Attention of one new token per sequence over the paged key/value pool (the
// pool that qkv_prologue_pool_write fills), split over the keys.
//
// A key's 4 D bytes (k and v of one head) meet 4 D G flops, G = n_q / n_kv query
// heads of the group: with G of 4 to 16 that is far below what the tensor cores
// could do, so the kernel is bound by reading the pool once, and its work is to
// keep enough of it in flight. Every warp is a worker of its own: it streams
// tiles of 16 keys of one key/value head through its own ring of shared memory
// (16-byte asynchronous copies, no barrier with other warps), with
//     S [16 heads x 16 keys] = Q K^T,  P = 2^(c S - m),  O += P V
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
#include "attention.cuh"

namespace qkvp {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kTileKeys = 16;

template <int HD>
struct DecSmem {
  static constexpr int kTileBytes = 2 * kTileKeys * HD * 2;  // k rows, then v rows
  static constexpr int kStages = HD == 128 ? 3 : 6;
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

// Keys of sequence b: the prefix (when it is not computed apart), then its own.
__device__ __forceinline__ int64_t dec_own(const AttnDecodeArgs& a, int b) {
  const int64_t n = a.lengths[b], most = (int64_t)a.max_pages * a.page_size;
  return n < 0 ? 0 : (n > most ? most : n);
}
__device__ __forceinline__ int dec_tiles(const AttnDecodeArgs& a, int b) {
  return (int)((a.joint_len + dec_own(a, b) + kTileKeys - 1) / kTileKeys);
}

// Whole warp: all tiles of the batch, and those of the sequences before `b`.
__device__ __forceinline__ int64_t dec_total(const AttnDecodeArgs& a, int b, int lane, int64_t* before) {
  int64_t all = 0, pre = 0;
  for (int s = lane; s < a.batch; s += 32) {
    const int n = dec_tiles(a, s);
    all += n;
    if (s < b) pre += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
  }
  *before = pre;
  return all;
}

__device__ __forceinline__ int64_t dec_quota(const AttnDecodeArgs& a, int64_t total) {
  const int64_t q = (total + a.ranges - 1) / a.ranges;
  return q < kDecMinTiles ? kDecMinTiles : q;
}

// A position in the concatenated tiles.
struct DecCursor {
  int b;      // sequence
  int tile;   // tile of it
  int tiles;  // its tiles
  __device__ __forceinline__ void settle(const AttnDecodeArgs& a) {
    while (tile >= tiles && b + 1 < a.batch) {
      tile -= tiles;
      ++b;
      tiles = dec_tiles(a, b);
    }
  }
};

// Pool row of key `key` of sequence b, or -1 (behind its end, or a bad page).
__device__ __forceinline__ int64_t dec_slot(const AttnDecodeArgs& a, int b, int64_t keys, int64_t key) {
  if (key >= keys) return -1;
  const int32_t* pages = a.prefix_pages;
  if (key >= a.joint_len) {
    key -= a.joint_len;
    pages = a.page_table + (int64_t)b * a.table_stride;
  }
  const int64_t p = key / a.page_size;
  const int page = pages[p];
  if (page < 0 || page >= a.num_pages) {
    if (a.dev_status) atomicOr(a.dev_status, kDevBadPage);
    return -1;
  }
  return (int64_t)page * a.page_size + (key - p * a.page_size);
}

}  // namespace

template <int HD>
__global__ void __launch_bounds__(kDecThreads, 1) qkvp_attention_decode_kernel(const AttnDecodeArgs a) {
  using SM = DecSmem<HD>;
  constexpr int ST = SM::kStages, CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks per row, rows per copy instruction
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ uint32_t s_in[kDecWarps][ST];  // bit i: key i of the stage's tile is attended
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_addr(smem_raw) + warp * SM::kWarpBytes;
  griddep_wait();
  griddep_launch_dependents();

  int64_t before;
  const int64_t total = dec_total(a, 0, lane, &before);
  const int64_t quota = dec_quota(a, total);
  const int heads = a.n_kv * a.head_blocks;
  const int64_t items = (int64_t)a.ranges * heads;
  for (int64_t w = (int64_t)blockIdx.x * kDecWarps + warp; w < items; w += (int64_t)gridDim.x * kDecWarps) {
    const int64_t range = w / heads, t0 = range * quota, t1 = min(total, t0 + quota);
    if (t0 >= t1) break;
    const int hv = (int)(w % heads), kvh = hv / a.head_blocks, hb = hv % a.head_blocks;
    const int head0 = kvh * a.group + hb * kTileKeys, n_heads = min(kTileKeys, a.group - hb * kTileKeys);

    // where the range begins
    DecCursor c{0, 0, 0};
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
          c.b = s0 + src;
          c.tiles = __shfl_sync(0xffffffffu, n, src);
          c.tile = (int)(left - (__shfl_sync(0xffffffffu, sum, src) - c.tiles));
          break;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
      }
    }

    // Loads run ST - 1 tiles ahead of the arithmetic, and the page lookup of a
    // tile one step ahead of its loads.
    DecCursor ld = c;
    int64_t ld_keys = a.joint_len + dec_own(a, ld.b), slot = -1;
    auto look_up = [&]() {
      if (lane < kTileKeys) slot = dec_slot(a, ld.b, ld_keys, (int64_t)ld.tile * kTileKeys + lane);
    };
    auto advance = [&]() {
      const int b = ld.b;
      ++ld.tile;
      ld.settle(a);
      if (ld.b != b) ld_keys = a.joint_len + dec_own(a, ld.b);
    };
    auto issue = [&](uint32_t st) {
      const uint32_t in = __ballot_sync(0xffffffffu, lane < kTileKeys && slot >= 0);
      if (lane == 0) s_in[warp][st] = in;
      const uint32_t dst = ring + st * SM::kTileBytes;
      const int ch = lane % CH;
#pragma unroll
      for (int i = 0; i < kTileKeys / RPI; ++i) {
        const int r = i * RPI + lane / CH;
        const int64_t row = __shfl_sync(0xffffffffu, slot, r);
        const int64_t off = ((row < 0 ? 0 : row) * a.n_kv + kvh) * CH + ch;
        const uint32_t to = dst + r * (HD * 2) + ((ch ^ (r & 7)) << 4);
        cp_async16(to, a.k_pool + off, row >= 0);
        cp_async16(to + kTileKeys * HD * 2, a.v_pool + off, row >= 0);
      }
    };
    const int64_t n_tiles = t1 - t0;
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
    float o[HD / 8][4], m[2], l[2];
    auto begin = [&]() {  // a sequence's first tile here
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = (lane >> 2) + 8 * (x & 1), d = 16 * ks + 8 * (x >> 1) + 2 * (lane & 3);
          qf[ks][x] = r < n_heads ? *reinterpret_cast<const uint32_t*>(
                                        a.q + ((int64_t)c.b * a.n_q + head0 + r) * HD + d)
                                  : 0u;
        }
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    };
    bool first = c.tile == 0;  // of the sequence: else the segment continues one of the range before
    auto end = [&]() {         // its last tile here: the partial result
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = (lane >> 2) + 8 * x;
        if (r < n_heads) {
          const int64_t row = (first ? (int64_t)c.b : a.batch + range) * a.n_q + head0 + r;
          if ((lane & 3) == 0) a.part_ml[row] = make_float2(m[x], l[x]);
          float2* dst = reinterpret_cast<float2*>(a.part_o + row * HD) + (lane & 3);
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) dst[4 * i] = make_float2(o[i][2 * x], o[i][2 * x + 1]);
        }
      }
    };
    begin();
    uint32_t st = 0;
    for (int64_t t = 0; t < n_tiles; ++t) {
      cp_wait<ST - 2>();
      __syncwarp();  // this tile is here, and every lane is done with the one before
      {
        const uint32_t nst = st == 0 ? ST - 1 : st - 1;
        if (t + ST - 1 < n_tiles) {
          issue(nst);
          if (t + ST < n_tiles) {
            advance();
            look_up();
          }
        }
        cp_commit();
      }
      const uint32_t kt = ring + st * SM::kTileBytes, vt = kt + kTileKeys * HD * 2;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int key = ((lane >> 4) << 3) + (lane & 7), hi = (lane >> 3) & 1;
        const uint32_t row = kt + key * (HD * 2);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          uint32_t b[4];
          ldsm4(row + (((2 * ks + hi) ^ (key & 7)) << 4), b);
          mma16816(s[0], qf[ks], b[0], b[1]);
          mma16816(s[1], qf[ks], b[2], b[3]);
        }
      }
      const uint32_t in = s_in[warp][st];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 8 * n + 2 * (lane & 3) + (x & 1);
          s[n][x] = (in >> key) & 1 ? s[n][x] * a.scale_log2 : -INFINITY;
        }
      float top[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        top[x] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      }
      // rescale only where a maximum grew by more than 8 powers of two (see the prompt kernel)
      if (__any_sync(0xffffffffu, top[0] - m[0] > 8.f || top[1] - m[1] > 8.f)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float m_new = fmaxf(m[x], top[x]);
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
      uint32_t pf[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float off = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(s[n][2 * x] - off), p1 = ex2(s[n][2 * x + 1] - off);
          l[x] += p0 + p1;
          pf[2 * n + x] = pack2(p0, p1);
        }
      }
      {
        const int key = (((lane >> 3) & 1) << 3) + (lane & 7), hi = lane >> 4;
        const uint32_t row = vt + key * (HD * 2);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          uint32_t b[4];
          ldsm4t(row + (((2 * i + hi) ^ (key & 7)) << 4), b);
          mma16816(o[2 * i], pf, b[0], b[1]);
          mma16816(o[2 * i + 1], pf, b[2], b[3]);
        }
      }
      st = st + 1 == ST ? 0 : st + 1;
      if (c.tile + 1 == c.tiles || t + 1 == n_tiles) {
        end();
        ++c.tile;
        c.settle(a);
        first = true;
        if (t + 1 < n_tiles) begin();
      } else {
        ++c.tile;
      }
    }
    cp_wait<0>();
    __syncwarp();
  }
}

// Joins the partial results of each (sequence, head): its own in the ranges it
// lies in and the shared prefix's key ranges, in that order. kJoinWarps warps per
// CTA, `wph` of them per head.
template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) qkvp_attention_join_kernel(const AttnDecodeArgs a) {
  constexpr int V = HD / 32;  // values per lane
  __shared__ float s_o[kJoinWarps][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = kJoinWarps / a.wph;  // heads per CTA
  const int groups = (a.n_q + per - 1) / per;
  const int b = (int)(blockIdx.x / groups), head = (int)(blockIdx.x % groups) * per + warp / a.wph;
  const int sub = warp % a.wph;
  griddep_wait();
  griddep_launch_dependents();
  int64_t before;
  const int64_t quota = dec_quota(a, dec_total(a, b, lane, &before));
  const int tiles = dec_tiles(a, b);
  if (threadIdx.x == 0 && blockIdx.x % groups == 0 && a.dev_status &&
      (a.lengths[b] < 0 || a.lengths[b] > (int64_t)a.max_pages * a.page_size))
    atomicOr(a.dev_status, kDevBadLength);
  const int64_t r0 = before / quota, r1 = tiles ? (before + tiles - 1) / quota : r0;
  const int own = tiles ? (int)(r1 - r0) + 1 : 0, parts = own + a.prefix_chunks;
  const bool on = head < a.n_q;
  // row of partial result i in part_o / part_ml: [batch] first pieces, [ranges] later ones, [prefix chunks][batch]
  auto row_of = [&](int i) -> int64_t {
    const int64_t r = i == 0 && own ? (int64_t)b
                      : i < own     ? a.batch + r0 + i
                                    : (int64_t)a.batch + a.ranges + (int64_t)(i - own) * a.batch + b;
    return r * a.n_q + head;
  };
  float top = -INFINITY, sum = 0.f, o[V] = {};
  if (on) {
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, a.part_ml[row_of(i)].x);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float off = top == -INFINITY ? 0.f : top;
    for (int i = lane; i < parts; i += 32) {
      const float2 v = a.part_ml[row_of(i)];
      sum += ex2(v.x - off) * v.y;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
#pragma unroll 4
    for (int i = sub; i < parts; i += a.wph) {
      const int64_t r = row_of(i);
      const float f = ex2(a.part_ml[r].x - off);
      const float* src = a.part_o + r * HD + V * lane;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(f, src[e], o[e]);
    }
  }
  if (a.wph > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][V * lane + e] = o[e];
    __syncthreads();
    if (sub == 0)
      for (int x = 1; x < a.wph; ++x)
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += s_o[warp + x][V * lane + e];
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
  return kDecWarps * (head_dim == 64 ? DecSmem<64>::kWarpBytes : DecSmem<128>::kWarpBytes);
}
int attention_decode_threads() { return kDecThreads; }
int attention_decode_warps() { return kDecWarps; }

}  // namespace qkvp
