// Attention forward on the tensor cores (sm_103a), for two callers:
//
//   prompt   causal attention over packed sequences: q [T, n_q, D], k and v
//            [T, n_kv, D], offsets cu[batch + 1]; writes out (bf16) and, for
//            training, the log-sum-exp of each row;
//   prefix   the query rows of a decode batch (sequence b, head g of the group
//            of key/value head h) against a prefix that all sequences share,
//            read from the paged pool; writes float32 partial results of key
//            ranges that the decode's last kernel joins.
//
// With s_ij = scale q_i . k_j over the keys row i may see,
//   m_i = max_j s_ij,  l_i = sum_j e^(s_ij - m_i),  o_i = sum_j e^(s_ij - m_i) v_j / l_i,
// in one pass over the keys, m and l running: a block of 128 keys gives S = Q K^T
// (fp32 in tensor memory), each row's maximum, P = e^(S - m) rounded to bf16 (the
// rounding of an operand of the second product; l sums P before it), and
// O += P V. When a row's maximum grows, what O and l hold has the factor
// e^(m_old - m_new). O is only rescaled when that maximum grew by more than 8
// powers of two: up to there P stays below 2^8, where bf16 has the same relative
// precision and the fp32 sums have room, and the division by l makes the
// reference point drop out.
//
// One CTA per SM holds two blocks of 128 query rows ("slots") that share every
// key block: two heads of the same group at the same rows where the group is
// even, else two consecutive row blocks of a head. Of a sequence of at most 64 (32) rows a
// slot holds two (four) heads of the group: a block costs a CTA some 6700
// cycles however few of its rows are there (60 sequences of 67 rows, 128 over 16 heads of
// 64: 122 us with a head a slot, 92 so when that was built). Sharing halves what K and V
// cost to fetch (64 KiB per 2 x 8.4 MFLOP at head_dim 128), and while one slot's
// softmax runs, the tensor cores work on the other's products:
//   warp 0      loads Q, K, V tiles with TMA into 128B-swizzled shared memory;
//   warp 1      issues the MMAs: PV(i) then S(i + 1) of slot 0, the same of slot 1. At
//               head_dim 128 P lives in the tensor-memory columns of the S it came
//               from; MMAs execute in order, so S(i + 1) overwrites P(i) after PV(i)
//               read it. At head_dim 64 there is room for P apart, and S(i + 1) is
//               issued as soon as the softmax has S(i) in registers. (One issuer per
//               slot measured slower, 1279 -> 1434 us at 16384 tokens and head_dim
//               128: the slots fall into step and their products collide.);
//   warp 2      finds the next work item (AttnOrder), one ahead, and at last zeroes the
//               rows of no sequence where the caller asked for it;
//   warps 4-7   softmax, rescaling and epilogue of slot 0, thread i owning row i,
//   warps 8-11  the same of slot 1.
// Keys behind the end of a sequence may hold anything (another sequence, unused
// memory): their scores are replaced, not added to, and their V rows are zeroed
// in shared memory, since 0 times a NaN is not 0.
//
// Measured: 16384 tokens, 32 over 8 heads of 128: 1356 us, 1622 TFLOP/s (0.85 of a large
// library product's burst rate), tensor pipe 68 % active; what is missing is the time
// between a block's scores and its weights, with registers and tensor memory full at two
// blocks. 8192 tokens in 23 sequences, 64 over 8 heads of 64: 93 us, bound by the chain of
// steps that a block of few keys goes through (some 3900 cycles a pair of blocks). The
// prefix of 32768 keys for 64 sequences, 32 over 8 heads of 128: 35 us (134 MB, 34 GFLOP),
// 13 of them ramp-up and results.
#include "attention.cuh"

namespace qkvp {
namespace {

constexpr int kFwdThreads = 384;
constexpr int kFwdSched = 2;  // work items in flight between the finder and the others
constexpr int kStageBytes = 32 * 128;  // an epilogue warp's buffer: 32 rows x 64 bf16
constexpr float kRescale = 8.f;  // powers of two a row's maximum may grow before O is rescaled

template <int HD>
struct FwdSmem {
  static constexpr int kTile = (HD / 64) * kAttnBox;  // 128 rows x HD bf16
  static constexpr int kStages = HD == 128 ? 4 : 8;  // K and V tiles in flight
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kOut = kRing + kStages * kTile;
  // tensor memory of slot j: scores, weights, result
  static constexpr bool kApart = HD == 64;  // P has its own columns
  __host__ __device__ static constexpr uint32_t tS(int j) { return kApart ? 256 * j : 128 * j; }
  __host__ __device__ static constexpr uint32_t tP(int j) { return kApart ? 256 * j + 128 : tS(j); }
  __host__ __device__ static constexpr uint32_t tO(int j) { return kApart ? 256 * j + 192 : 256 + 128 * j; }
};

struct FwdItem {
  int n0, n1;        // key blocks of each slot (0: the slot is idle)
  int row0, row1;    // first query row of each slot (prompt: of T; prefix: row tile)
  int head0, head1;  // query head of each slot
  int kvh;           // key/value head
  int kv0;           // first key row (prompt)
  int len;           // keys (of the sequence, or of this key range of the prefix)
  int hs;            // prompt: heads in a tile, as in attn_load_tile
  int end;           // prompt: end of the group's query heads (a tile may have room for more)
  int valid;
};

}  // namespace

template <int HD, bool PREFIX>
__global__ void __launch_bounds__(kFwdThreads, 1)
    qkvp_attention_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                              const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap pieces_q,
                              const AttnFwdArgs a) {
  using SM = FwdSmem<HD>;
  constexpr int ST = SM::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[ST], empty[ST], tail_bar, mma_done, q_full[2], q_empty[2], s_full[2],
      s_read[2], p_full[2], o_done[2], o_free[2], it_full[kFwdSched], it_empty[kFwdSched];
  __shared__ uint32_t s_tmem;
  __shared__ AttnWatch s_watch;
  __shared__ FwdItem s_item[kFwdSched];
  __shared__ int s_cache[PREFIX ? 1 : AttnOrder::kCached];
  __shared__ int s_slot[PREFIX ? kAttnMaxChunk / 8 : 1];  // pool row of each page box of the key range, or -1
  __shared__ uint32_t s_whole;                            // prefix: bit i set when all 128 keys of block i are valid
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tail_bar, 1);
    mbar_init(&mma_done, 1);
    for (int j = 0; j < 2; ++j) {
      mbar_init(&q_full[j], 1);
      mbar_init(&q_empty[j], 1);
      mbar_init(&s_full[j], 1);
      mbar_init(&s_read[j], 4);
      mbar_init(&p_full[j], 4);
      mbar_init(&o_done[j], 1);
      mbar_init(&o_free[j], 4);
    }
    for (int j = 0; j < kFwdSched; ++j) {
      mbar_init(&it_full[j], 1);
      mbar_init(&it_empty[j], 10);  // loader, issuer, 8 softmax warps
    }
    s_watch.fail = 0;
    s_whole = 0xffffffffu;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(&s_tmem, 512);
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x == 0) attn_beat(&s_watch);  // (not before: the launches before this one may take any time)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = attn_wait(bar, parity, &s_watch);
    __syncwarp();
    return ok;
  };

  int px_len = 0, px_first = 0, px_chunk = 0;  // prefix: this CTA's key range
  if constexpr (PREFIX) {
    const int per = a.n_kv * a.pairs;
    px_chunk = (int)blockIdx.x / per;
    px_first = px_chunk * a.chunk;
    px_len = min(a.chunk, a.prefix_len - px_first);
    const int boxes = (px_len + a.box_rows - 1) / a.box_rows;
    for (int g = threadIdx.x; g < boxes; g += kFwdThreads) {
      const int key = px_first + g * a.box_rows;
      const int page = a.prefix_pages[key / a.page_size];
      const bool ok = page >= 0 && page < a.num_pages;
      s_slot[g] = ok ? page * a.page_size + key % a.page_size : -1;
      if (!ok) {
        atomicAnd(&s_whole, ~(1u << (g * a.box_rows / kAttnRows)));
        if (a.dev_status) atomicOr(a.dev_status, kDevBadPage);
      }
    }
    if (threadIdx.x == 0 && px_len % kAttnRows) atomicAnd(&s_whole, ~(1u << (px_len / kAttnRows)));
    __syncthreads();
  }

  // The next work item, in order: read from the finder's ring, or (prefix) the
  // CTA's only one. Every role sees the same items.
  uint32_t it_pos = 0;
  auto next_item = [&](FwdItem& t) -> bool {
    if constexpr (PREFIX) {
      if (it_pos++) return false;
      const int r = (int)blockIdx.x % (a.n_kv * a.pairs);
      t.kvh = r % a.n_kv;
      const int n = (px_len + kAttnRows - 1) / kAttnRows;
      t.row0 = 2 * (r / a.n_kv);
      t.row1 = t.row0 + 1;
      t.n0 = n;
      t.n1 = t.row1 < a.row_tiles ? n : 0;
      t.head0 = t.head1 = 0;
      t.kv0 = 0;
      t.len = px_len;
      return true;
    } else {
      const uint32_t s = it_pos % kFwdSched, ph = (it_pos / kFwdSched) & 1;
      ++it_pos;
      if (!__all_sync(0xffffffffu, wait(&it_full[s], ph))) return false;
      t = s_item[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[s]);
      return t.valid != 0;
    }
  };

  // 12 warps launched with 168 registers a thread (the launch bounds' share of 65536):
  // 4 warps x 88 + 8 x 208 = 12 x 168. A softmax thread holds its row's 128 scores.
  if (warp < 4) {
    regs_less<88>();
    if (warp == 0) {
      // ---- loader. A wait for a buffer that was never used passes: the phase before a
      // barrier's first counts as complete.
      uint32_t it = 0, tails = 0, q_ph = 0;  // ring position; bit j: phase of slot j's query tile
      FwdItem t;
      while (next_item(t)) {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          if ((j ? t.n1 : t.n0) == 0) continue;
          wait(&q_empty[j], ((q_ph >> j) & 1) ^ 1);
          q_ph ^= 1u << j;
          unsigned char* dst = base + SM::kQ + j * SM::kTile;
          const int row = j ? t.row1 : t.row0, head = j ? t.head1 : t.head0;
          if (lane == 0)
            mbar_arrive_expect_tx(&q_full[j], PREFIX ? (uint32_t)(a.bpt * a.group * HD * 2) : (uint32_t)SM::kTile);
          __syncwarp();
          if constexpr (!PREFIX)
            attn_load_tile<HD>(dst, &tmap_q, &pieces_q, head * HD, row, t.hs, &q_full[j], lane);
          else if (lane < HD / 64)
            tma_load_3d(dst + lane * kAttnBox, &tmap_q, 64 * lane, t.kvh * a.group, row * a.bpt, &q_full[j]);
        }
        const int n = max(t.n0, t.n1);
#pragma unroll 1
        for (int i2 = 0; i2 < 2 * n; ++i2, ++it) {  // K and V of block 0, of block 1, ...
          const int i = i2 >> 1, which = i2 & 1;
          const uint32_t s = it % ST;
          wait(&empty[s], ((it / ST) & 1) ^ 1);
          if (lane == 0) attn_beat(&s_watch);
          unsigned char* dst = base + SM::kRing + s * SM::kTile;
          const CUtensorMap* map = which ? &tmap_v : &tmap_k;
          const bool part = PREFIX ? ((s_whole >> i) & 1) == 0 : kAttnRows * (i + 1) > t.len;
          const bool patch = which && part;  // rows of V to zero once they are here
          uint64_t* bar = patch ? &tail_bar : &full[s];
          if constexpr (PREFIX) {
            // one box per page piece (box_rows keys); lanes take them in turn
            const int per = kAttnRows / a.box_rows;
            const int gg = i * per + lane;  // box_rows >= 8: at most 16 pieces
            const bool mine = lane < per && gg * a.box_rows < px_len && s_slot[gg] >= 0;
            const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * a.box_rows * HD * 2));
            __syncwarp();
            if (mine)
#pragma unroll
              for (int x = 0; x < HD / 64; ++x)
                tma_load_3d(dst + x * kAttnBox + lane * a.box_rows * 128, map, 64 * x, t.kvh, s_slot[gg], bar);
          } else if (lane == 0) {
            mbar_arrive_expect_tx(bar, SM::kTile);
#pragma unroll
            for (int x = 0; x < HD / 64; ++x)
              tma_load_2d(dst + x * kAttnBox, map, t.kvh * HD + 64 * x, t.kv0 + kAttnRows * i, bar);
          }
          if (patch) {
            wait(&tail_bar, tails++ & 1);
#pragma unroll 1
            for (int r = lane >> 3; r < kAttnRows; r += 4) {
              const int key = kAttnRows * i + r;
              if (key < t.len && (!PREFIX || s_slot[key / a.box_rows] >= 0)) continue;
#pragma unroll
              for (int x = 0; x < HD / 64; ++x)
                *reinterpret_cast<uint4*>(dst + x * kAttnBox + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
          }
        }
      }
      // every copy has landed before the CTA may exit (phases already consumed return at once)
      if (lane == 0) {
#pragma unroll 1
        for (uint32_t k = it > ST ? it - ST : 0; k < it; ++k) mbar_wait(&full[k % ST], (k / ST) & 1, a.err);
        // slot j's last query tile: its phase is the one before the next
#pragma unroll 1
        for (int j = 0; j < 2; ++j) mbar_wait(&q_full[j], ((q_ph >> j) & 1) ^ 1, a.err);
      }
    } else if (warp == 1) {
      // ---- MMA issuer. Step i: P V of block i and the scores of block i + 1.
      constexpr uint32_t id_s = umma_idesc_bf16(kAttnRows, kAttnRows), id_o = umma_idesc_bf16_bmn(kAttnRows, HD);
      uint32_t it = 0, q_ph = 0, p_ph = 0, o_ph = 0;  // bit j: phases of slot j
      const uint32_t tmem = uniform(s_tmem);
      FwdItem t;
      while (next_item(t)) {
        const int n0 = (int)uniform(t.n0), n1 = (int)uniform(t.n1), n = max(n0, n1);
        auto tile = [&](uint32_t k) { return base + SM::kRing + (k % ST) * SM::kTile; };
        auto scores = [&](int j, int i, int nj) {
          if (i == 0) {
            wait(&q_full[j], (q_ph >> j) & 1);
            q_ph ^= 1u << j;
          }
          tc_fence_after();
          attn_mma_ss<HD>(tmem + SM::tS(j), base + SM::kQ + j * SM::kTile, tile(it + 2 * i), id_s);
          umma_commit_warp(&s_full[j]);
          if (i + 1 == nj) umma_commit_warp(&q_empty[j]);
        };
#pragma unroll 1
        for (int i = -1; i < n; ++i) {
          const uint32_t kv = it + 2 * i + 1, kn = it + 2 * i + 2;
          if (i + 1 < n) wait(&full[kn % ST], (kn / ST) & 1);
          if (SM::kApart && i + 1 < n) {  // the next scores as soon as the last ones have been read
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int nj = j ? n1 : n0;
              if (i + 1 >= nj) continue;
              if (i >= 0) wait(&s_read[j], (p_ph >> j) & 1);
              scores(j, i + 1, nj);
            }
            umma_commit_warp(&empty[kn % ST]);
          }
          if (i >= 0) wait(&full[kv % ST], (kv / ST) & 1);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int nj = j ? n1 : n0;
            if (i >= 0 && i < nj) {
              wait(&p_full[j], (p_ph >> j) & 1);
              p_ph ^= 1u << j;
              if (i == 0) {
                wait(&o_free[j], ((o_ph >> j) & 1) ^ 1);
                o_ph ^= 1u << j;
              }
              tc_fence_after();
              attn_mma_ts(tmem + SM::tO(j), tmem + SM::tP(j), 32, tile(kv), id_o, i > 0);
              umma_commit_warp(&o_done[j]);
            }
            if (!SM::kApart && i + 1 < nj) scores(j, i + 1, nj);
          }
          if (i >= 0) umma_commit_warp(&empty[kv % ST]);
          if (!SM::kApart && i + 1 < n) umma_commit_warp(&empty[kn % ST]);
        }
        it += 2 * n;
      }
      umma_commit_warp(&mma_done);  // nothing it issued may still run when the CTA exits
      if (lane == 0) mbar_wait(&mma_done, 0, a.err);
    } else if (warp == 2 && !PREFIX) {
      // ---- finder
      AttnOrder ord{a.cu, a.batch, a.pair_heads ? kAttnRows : 2 * kAttnRows, (uint32_t)a.units, (uint32_t)a.units64,
                    (uint32_t)a.units32, s_cache};
      const bool good = ord.init(a.T, lane);
      if (!good && blockIdx.x == 0 && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDevBadSequence);
      const uint32_t work = ord.work();  // below 2^31: the host checks
      for (uint32_t k = 0;; ++k) {
        const uint32_t s = k % kFwdSched;
        if (!__all_sync(0xffffffffu, wait(&it_empty[s], ((k / kFwdSched) & 1) ^ 1))) break;
        const uint32_t w = attn_deal(k, blockIdx.x, gridDim.x);
        FwdItem t = {};
        t.valid = k * gridDim.x < work;  // else no CTA has any left
        if (w < work) {                  // (an empty item: this CTA has none in the last round)
          int seq, cost, hu;
          ord.find(w, lane, seq, cost, hu, t.hs);
          const int start = a.cu[seq], len = a.cu[seq + 1] - start;
          if (t.hs != 2) {  // a slot holds up to 4 >> hs heads of the group
            const int items = (t.hs ? a.units64 : a.units32) / a.n_kv, kvh = hu / items;
            t.head0 = kvh * a.group + (hu - kvh * items) * (8 >> t.hs);
            t.head1 = t.head0 + (4 >> t.hs);
            t.row0 = t.row1 = start;
            t.n0 = 1;
            t.n1 = t.head1 < (kvh + 1) * a.group;
          } else if (a.pair_heads) {
            t.head0 = 2 * hu;
            t.head1 = t.head0 + 1;
            t.row0 = t.row1 = start + kAttnRows * (cost - 1);
            t.n0 = t.n1 = cost;
          } else {
            t.head0 = t.head1 = hu;
            t.row0 = start + 2 * kAttnRows * (cost - 1);
            t.row1 = t.row0 + kAttnRows;
            t.n0 = 2 * cost - 1;
            t.n1 = t.row1 < start + len ? 2 * cost : 0;
          }
          t.kvh = t.head0 / a.group;
          t.end = (t.kvh + 1) * a.group;
          t.kv0 = start;
          t.len = len;
        }
        if (lane == 0) {
          s_item[s] = t;
          mbar_arrive(&it_full[s]);
        }
        __syncwarp();
        if (!t.valid) break;
      }
      // ---- then the rows of no sequence
      if (a.zero_rest) {
        const bool none = !good || a.batch == 0;
        const int64_t first = none ? 0 : a.cu[0], last = none ? 0 : a.cu[a.batch];
        attn_zero_rows(a.out, a.T, a.n_q * (HD / 8), first, last, lane);
        if (a.lse)
#pragma unroll 1
          for (int h = blockIdx.x; h < a.n_q; h += gridDim.x)
#pragma unroll 1
            for (int64_t r = lane; r < first + a.T - last; r += 32)
              a.lse[h * a.T + (r < first ? r : last + (r - first))] = -INFINITY;
      }
    }
  } else {
    regs_more<208>();
    // ---- softmax, rescaling, results
    const int j = (warp - 4) >> 2, qtr = warp & 3, row = 32 * qtr + lane;
    const uint32_t lanes = (uint32_t)(32 * qtr) << 16;
    const uint32_t t_s = tmem + lanes + SM::tS(j), t_p = tmem + lanes + SM::tP(j), t_o = tmem + lanes + SM::tO(j);
    const float c = a.scale_log2;
    uint32_t done = 0;  // blocks of this slot so far
    FwdItem t;
    while (next_item(t)) {
      const int n = j ? t.n1 : t.n0;
      if (n == 0) continue;
      // this warp's 32 rows of its head's (PREFIX: hs plays no part)
      const int vq = PREFIX ? qtr : qtr & ((1 << t.hs) - 1);
      const int row0 = (j ? t.row1 : t.row0) + 32 * vq;
      const int head = (j ? t.head1 : t.head0) + (PREFIX ? 0 : qtr >> t.hs);
      // prompt: rows of this warp that belong to the sequence
      const int rows = PREFIX || head < t.end ? t.kv0 + t.len - row0 : 0;
      // A row of something else (another sequence, unused memory) has no say in when its warp
      // rescales: that would show in the other rows' last bits.
      const bool live = PREFIX ? row < a.bpt * a.group : lane < rows;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++done) {
        wait(&s_full[j], done & 1);
        tc_fence_after();
        if (!PREFIX && rows <= 0) {  // whatever P holds for rows of no sequence stays in those rows
          if (SM::kApart) {
            if (lane == 0) mbar_arrive(&s_read[j]);
            if (i > 0) wait(&o_done[j], (done - 1) & 1);  // not two blocks' arrivals in one phase of p_full
          }
          if (lane == 0) mbar_arrive(&p_full[j]);
          continue;
        }
        float s[kAttnRows];
        float top = tmem_ld128_max(t_s, s);
        if constexpr (SM::kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_read[j]);
        }
        int quarters = 4;  // 32-key quarters of the block that any row of this warp sees
        if constexpr (PREFIX) {
          if (!((s_whole >> i) & 1)) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = kAttnRows * i + 32 * x + lane;
              const uint32_t in =
                  __ballot_sync(0xffffffffu, key < px_len && s_slot[min(key, px_len - 1) / a.box_rows] >= 0);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((in >> e) & 1)) s[32 * x + e] = -INFINITY;
            }
            top = fmaxf(fmaxf(max32(s), max32(s + 32)), fmaxf(max32(s + 64), max32(s + 96)));
          }
        } else if (i == n - 1) {
          // the diagonal block: keys after the row (and so behind the sequence) are not
          // seen. The warp's rows see the quarters before their own whole, their own up
          // to the lane, and none after it. (The empty asm makes a branch of each quarter:
          // selects run at half rate, and all 128 of them took longer than the exponentials.)
          quarters = vq + 1;
          top = -INFINITY;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (x == vq) {
              asm volatile("");
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > lane) s[32 * x + e] = -INFINITY;
            }
            if (x <= vq) {
              asm volatile("");
              top = fmaxf(top, max32(s + 32 * x));
            }
          }
        }
        if (i == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, live && (top - m) * c > kRescale)) {  // also where m is -inf and top is not
          const float m_new = fmaxf(m, top);
          const float f = m_new == m ? 1.f : ex2((m - m_new) * c);
          m = m_new;
          l *= f;
          wait(&o_done[j], (done - 1) & 1);
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < HD; x += 16) tmem_scale16(t_o + x, f);
        }
        const float off = m == -INFINITY ? 0.f : -m * c;
        if (SM::kApart && i > 0) wait(&o_done[j], (done - 1) & 1);  // PV before has read the columns that P goes to
        const uint64_t c2 = pair(c, c), off2 = pair(off, off);
        uint64_t sum_a = 0, sum_b = 0;  // pairs of zeros
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t w[16];
          if (!PREFIX && x >= quarters) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0;
          } else {
            asm volatile("");
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              unpair(fma2(pair(s[32 * x + 2 * e], s[32 * x + 2 * e + 1]), c2, off2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              if (e & 1)
                sum_b = add2(sum_b, pair(p0, p1));
              else
                sum_a = add2(sum_a, pair(p0, p1));
              w[e] = pack2(p0, p1);
            }
          }
          tmem_st16(t_p + 16 * x, w);
        }
        float sum0, sum1;
        unpair(add2(sum_a, sum_b), sum0, sum1);
        l += sum0 + sum1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[j]);
      }
      wait(&o_done[j], (done - 1) & 1);
      tc_fence_after();
      if constexpr (PREFIX) {
        // O through shared memory (the slot's query tile, which nothing reads any more), 32
        // columns at a time: whole 128-byte lines leave
        const int first = (j ? t.row1 : t.row0) * a.bpt;  // of the tile's sequences
        const int64_t part = ((int64_t)px_chunk * a.batch + first) * a.n_q + t.kvh * a.group;
        auto place = [&](int r) -> int64_t {  // result row of the tile's row r, or -1
          const int b = r / a.group;
          return b < a.bpt && first + b < a.batch ? part + (int64_t)b * a.n_q + (r - b * a.group) : -1;
        };
        const int64_t mine = place(row);
        if (mine >= 0) a.part_ml[mine] = make_float2(m * c, l);
        const int r0 = lane >> 3, ch0 = lane & 7;
        unsigned char* buf = base + SM::kQ + j * SM::kTile + qtr * kStageBytes;
#pragma unroll 1
        for (int x = 0; x < HD / 32; ++x) {
          float o[32];
          tmem_ld32(t_o + 32 * x, o);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(buf + attn_swz(lane, e)) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int r4 = 0; r4 < 8; ++r4) {
            const float4 v = *reinterpret_cast<const float4*>(buf + attn_swz(4 * r4 + r0, ch0));
            const int64_t at = __shfl_sync(0xffffffffu, mine, 4 * r4 + r0);
            if (at >= 0) reinterpret_cast<float4*>(a.part_o + at * HD)[8 * x + ch0] = v;
          }
          __syncwarp();
        }
      } else if (rows <= 0) {
        if (lane == 0) mbar_arrive(&o_free[j]);
      } else {
        // O / l through shared memory, 64 columns at a time, so that whole 128-byte lines
        // leave: eight lanes per row, four rows per store
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN stays one
        const int r0 = lane >> 3, ch0 = lane & 7;
        unsigned char* buf = base + SM::kOut + (warp - 4) * kStageBytes;
        const int64_t stride = (int64_t)a.n_q * (HD / 8);
        uint4* dst = a.out + (row0 + r0) * stride + head * (HD / 8) + ch0;
#pragma unroll 1
        for (int x = 0; x < HD / 64; ++x) {
          float o[64];
          tmem_ld32(t_o + 64 * x, o);
          tmem_ld32(t_o + 64 * x + 32, o + 32);
          if (x + 1 == HD / 64) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[j]);
          }
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const float* v = o + 8 * ch;
            *reinterpret_cast<uint4*>(buf + attn_swz(lane, ch)) =
                make_uint4(pack2(v[0] * inv, v[1] * inv), pack2(v[2] * inv, v[3] * inv), pack2(v[4] * inv, v[5] * inv),
                           pack2(v[6] * inv, v[7] * inv));
          }
          __syncwarp();
          uint4 w[8];
#pragma unroll
          for (int r4 = 0; r4 < 8; ++r4) w[r4] = *reinterpret_cast<const uint4*>(buf + attn_swz(4 * r4 + r0, ch0));
          __syncwarp();
#pragma unroll
          for (int r4 = 0; r4 < 8; ++r4)
            if (4 * r4 + r0 < rows) dst[4 * r4 * stride + 8 * x] = w[r4];
        }
        if (a.lse && lane < rows) a.lse[(int64_t)head * a.T + row0 + lane] = m * a.scale + logf(l);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  attn_report(&s_watch, a.err);
}

const void* attention_fwd_kernel(int head_dim, bool prefix) {
  if (head_dim == 64)
    return prefix ? reinterpret_cast<const void*>(&qkvp_attention_fwd_kernel<64, true>)
                  : reinterpret_cast<const void*>(&qkvp_attention_fwd_kernel<64, false>);
  return prefix ? reinterpret_cast<const void*>(&qkvp_attention_fwd_kernel<128, true>)
                : reinterpret_cast<const void*>(&qkvp_attention_fwd_kernel<128, false>);
}

int attention_fwd_smem_bytes(int head_dim, bool prefix) {
  return 1024 + (head_dim == 64 ? FwdSmem<64>::kOut : FwdSmem<128>::kOut) + (prefix ? 0 : 8 * kStageBytes);
}
int attention_fwd_threads() { return kFwdThreads; }

}  // namespace qkvp
