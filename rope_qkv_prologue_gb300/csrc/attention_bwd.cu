// Backward of the causal attention over packed sequences (sm_103a): dq, dk and
// dv from dout, the inputs and the forward's out and lse.
//
// With p_ij = e^(s_ij - lse_i), delta_i = dout_i . out_i, dp_ij = dout_i . v_j and
// ds_ij = p_ij (dp_ij - delta_i):
//     dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j,
// dk and dv summed over the query heads of the group too. Sequences of at most 64 (32)
// rows have two (four) heads of the group in a tile of 128 queries (25 tokens in 19
// sequences, 256 over 16 heads of 64, both directions: 183 -> 64 us). Two kernels:
//   1. the query kernel: a CTA owns 128 queries of one head and goes through its
//      keys, adding dS K. Its dout is in shared memory, so it also forms delta and
//      leaves it for the other (against a kernel of its own for delta, 4096 tokens in
//      11 sequences take the same time, 700 in 3 take 55 us instead of 65);
//   2. the key/value kernel: a CTA owns 128 keys of one key/value head and goes
//      through the query blocks and heads that attend them, forming the transposed
//      S^T = K Q^T and dP^T = V dO^T and adding P^T dO and dS^T Q. Where that leaves
//      SMs idle (few tokens, few key/value heads), a group's query heads are divided
//      among CTAs, whose fp32 sums the folding kernel adds in a fixed order.
// S and dP are formed twice (seven products instead of five), so that every result
// is a sum in tensor memory in a fixed order: no atomics, the same bits every time.
//
// Both kernels are one template: two tiles of the CTA's own rows stay in shared
// memory, pairs of tiles stream past them by TMA, X = A1 B1^T and Y = A2 B2^T go
// to tensor memory, 256 threads turn them into bf16 P and dS in tensor memory (in
// the columns they came from), and those are the first operands of the
// accumulating products. A thread owns a row and half of a block's columns. MMAs
// execute in order, so a product may be issued over an operand of the one before it.
// P and dS are rounded to bf16 as operands; all sums are fp32.
//   warp 0      loads tiles (and zeroes rows behind a sequence's end in those that
//               are summed over: 0 times whatever is there need not be 0);
//   warp 1      issues the MMAs;
//   warp 2      finds work items (AttnOrder), one ahead;
//   warp 3      key/value kernel: lse and delta of the streamed rows; query kernel:
//               zeros in the rows of no sequence, where the caller asked for them;
//   warps 4-11  the arithmetic between the products, and the results' stores.
//
// Measured: 8192 tokens, 32 over 8 heads of 128: query kernel 528 us, key/value kernel
// 655 us, tensor pipe 67 and 72 % active (1580 us with the forward, 1664 in a steady loop:
// 0.64 and 0.61 of the library rate in the five products that a backward needs). 4096 tokens
// in 11 sequences, 128 over 16 heads of 64: 167 and 152 us, tensor pipe 22 and 33 % active;
// some 3400 and 3100 cycles a block, with one block in flight: X, P, dP, dS and the products
// in turn, all eight warps on the same block.
#include "attention.cuh"

namespace qkvp {
namespace {

constexpr int kBwdThreads = 384;
constexpr int kBwdSched = 2;
constexpr int kStatStages = 2;
constexpr int kStageBytes = 32 * 64;  // a warp's store buffer: 32 rows x 32 bf16

// Shared memory. The first streamed operand stays until the accumulating product of
// its block, two products after the first use, so it has the deeper ring (with two
// tiles the query kernel at head_dim 128 waited 1500 of 2800 cycles a block for K).
// At head_dim 128 that fills the SM's 227 KiB, and the results are stored from
// registers; at 64 they pass through a buffer that makes whole sectors of them.
template <int HD>
struct BwdSmem {
  static constexpr int kTile = (HD / 64) * kAttnBox;
  static constexpr int kS1 = HD == 128 ? 3 : 4, kS2 = HD == 128 ? 2 : 4;  // tiles of each streamed operand
  static constexpr int kA = 0;
  static constexpr int kB1 = 2 * kTile;
  static constexpr int kB2 = kB1 + kS1 * kTile;
  static constexpr int kOut = kB2 + kS2 * kTile;
  static constexpr int kBytes = kOut + (HD == 128 ? 0 : 8 * kStageBytes);
};

struct BwdItem {
  int n;      // streamed blocks
  int own;    // first row of the CTA's own block, of T
  int first;  // first row of the sequence
  int len;    // its rows
  int blk;    // the own block's index in the sequence
  int head;   // key/value head, or query head
  int hs;     // heads in a tile of queries, as in attn_load_tile
  int end;    // end of the query heads (a tile may have room for more)
  int split;  // SPLIT: which of the group's parts of query heads
  int valid;
};

}  // namespace

// KV: the key/value kernel; SPLIT: of it, with the heads of a group divided (an instance
// of its own: the division inside the one kernel cost it a tenth on ragged sequences).
template <int HD, bool KV, bool SPLIT>
__global__ void __launch_bounds__(kBwdThreads, 1)
    qkvp_attention_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                              const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                              const __grid_constant__ CUtensorMap pieces_q,
                              const __grid_constant__ CUtensorMap pieces_do, const AttnBwdArgs a) {
  using SM = BwdSmem<HD>;
  constexpr int S1 = SM::kS1, S2 = SM::kS2;
  // Tensor memory. X has two buffers where there is room for them (not in the
  // key/value kernel at head_dim 128); a block's P lies over its X, and its dS in
  // the columns of X that P leaves free, or over Y where X has one buffer.
  constexpr bool kTwoX = !KV || HD == 64;
  constexpr uint32_t tX = 0, tY = kTwoX ? 256 : 128, tAcc1 = tY + 128, tAcc2 = tAcc1 + HD;
  constexpr bool kAhead = kTwoX && S1 >= 4;  // X is issued two blocks ahead: three streamed tiles in use
  constexpr uint32_t kDsOff = KV && kTwoX ? 32 : 0;  // columns of dS behind those of P, in each half
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw;  // all of the SM's shared memory at head_dim 128: no room to round it up
  if ((smem_addr(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrWaitTimeout);  // no result; the declared alignment rules it out
    return;
  }
  __shared__ __align__(8) uint64_t a_full, a_empty, b1_full[S1], b1_empty[S1], b2_full[S2], b2_empty[S2], tail_bar,
      x_full[2], y_full, p_full, ds_full, acc_done, acc_free, st_full[kStatStages], st_empty[kStatStages],
      it_full[kBwdSched], it_empty[kBwdSched], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ AttnWatch s_watch;
  __shared__ BwdItem s_item[kBwdSched];
  __shared__ int s_cache[AttnOrder::kCached];
  // key/value kernel: -lse log2(e) and -delta of the streamed rows; query kernel: the
  // halves' parts of a row's sums
  __shared__ __align__(16) float s_stat[KV ? kStatStages : 2][2][kAttnRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&a_full, 1);
    mbar_init(&a_empty, 1);
    for (int s = 0; s < S1; ++s) {
      mbar_init(&b1_full[s], 1);
      mbar_init(&b1_empty[s], 1);
    }
    for (int s = 0; s < S2; ++s) {
      mbar_init(&b2_full[s], 1);
      mbar_init(&b2_empty[s], 1);
    }
    mbar_init(&tail_bar, 1);
    mbar_init(&x_full[0], 1);
    mbar_init(&x_full[1], 1);
    mbar_init(&y_full, 1);
    mbar_init(&p_full, 8);
    mbar_init(&ds_full, 8);
    mbar_init(&acc_done, 1);
    mbar_init(&acc_free, 8);
    for (int s = 0; s < kStatStages; ++s) {
      mbar_init(&st_full[s], 1);
      mbar_init(&st_empty[s], 8);
    }
    for (int s = 0; s < kBwdSched; ++s) {
      mbar_init(&it_full[s], 1);
      mbar_init(&it_empty[s], KV ? 11 : 10);  // loader, issuer, 8 arithmetic warps, the statistics' loader
    }
    mbar_init(&mma_done, 1);
    s_watch.fail = 0;
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
  uint32_t it_pos = 0;
  auto next_item = [&](BwdItem& t) -> bool {
    const uint32_t s = it_pos % kBwdSched, ph = (it_pos / kBwdSched) & 1;
    ++it_pos;
    if (!__all_sync(0xffffffffu, wait(&it_full[s], ph))) return false;
    t = s_item[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_empty[s]);
    return t.valid != 0;
  };
  // Streamed block i of an item: its index in the sequence, and (key/value
  // kernel) the query head.
  auto block_of = [&](const BwdItem& t, int i, int& head) {
    if constexpr (KV) {
      const int heads = SPLIT ? a.group / a.splits : a.group, per = t.n / ((heads + (4 >> t.hs) - 1) >> (2 - t.hs));
      head = t.end - heads + ((i / per) << (2 - t.hs));
      return t.blk + i % per;
    } else {
      head = t.head / a.group;
      return i;
    }
  };

  // 12 warps launched with 168 registers a thread: 4 warps x 88 + 8 x 208 = 12 x 168
  if (warp < 4) {
    regs_less<88>();
    if (warp == 0) {
      // ---- loader
      uint32_t it = 0, tails = 0, items = 0;
      BwdItem t;
      while (next_item(t)) {
        if (t.n == 0) continue;
        if (items > 0) wait(&a_empty, (items - 1) & 1);
        ++items;
        if (lane == 0) mbar_arrive_expect_tx(&a_full, 2 * SM::kTile);
        __syncwarp();
        if constexpr (!KV) {
          attn_load_tile<HD>(base + SM::kA, &tmap_q, &pieces_q, t.head * HD, t.own, t.hs, &a_full, lane);
          attn_load_tile<HD>(base + SM::kA + SM::kTile, &tmap_do, &pieces_do, t.head * HD, t.own, t.hs, &a_full, lane);
        } else if (lane < HD / 64) {
          tma_load_2d(base + SM::kA + lane * kAttnBox, &tmap_k, t.head * HD + 64 * lane, t.own, &a_full);
          tma_load_2d(base + SM::kA + SM::kTile + lane * kAttnBox, &tmap_v, t.head * HD + 64 * lane, t.own, &a_full);
        }
        for (int i = 0; i < t.n; ++i, ++it) {
          int head;
          const int blk = block_of(t, i, head);
          const int rows = t.len - kAttnRows * blk;  // of the sequence in this block
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            const uint32_t n = which ? S2 : S1, s = it % n;
            uint64_t* full = which ? &b2_full[s] : &b1_full[s];
            wait(which ? &b2_empty[s] : &b1_empty[s], ((it / n) & 1) ^ 1);  // (the first time round it passes)
            if (lane == 0) attn_beat(&s_watch);
            unsigned char* dst = base + (which ? SM::kB2 : SM::kB1) + s * SM::kTile;
            const CUtensorMap* map = KV ? (which ? &tmap_do : &tmap_q) : (which ? &tmap_v : &tmap_k);
            const int piece = KV ? 32 << t.hs : kAttnRows;  // rows of a head in the tile
            const int held = KV ? piece * (t.end - head) : kAttnRows;  // rows of its heads (or more)
            const bool patch = (rows < piece || held < kAttnRows) && (KV || which == 0);
            uint64_t* bar = patch ? &tail_bar : full;
            if (lane == 0) mbar_arrive_expect_tx(bar, SM::kTile);
            __syncwarp();
            if constexpr (KV)
              attn_load_tile<HD>(dst, map, which ? &pieces_do : &pieces_q, head * HD, t.first + kAttnRows * blk, t.hs,
                                 bar, lane);
            else if (lane < HD / 64)
              tma_load_2d(dst + lane * kAttnBox, map, head * HD + 64 * lane, t.first + kAttnRows * blk, bar);
            if (patch) {
              wait(&tail_bar, tails++ & 1);
              for (int r = min(rows, held) + (lane >> 3); r < kAttnRows; r += 4)
                for (int x = 0; x < HD / 64 && ((r & (piece - 1)) >= rows || r >= held); ++x)
                  *reinterpret_cast<uint4*>(dst + x * kAttnBox + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_cta();
              __syncwarp();
              if (lane == 0) mbar_arrive(full);
            }
          }
        }
      }
      // every copy has landed before the CTA may exit (phases already consumed return at once)
      if (lane == 0) {
        for (uint32_t k = it > S1 ? it - S1 : 0; k < it; ++k) mbar_wait(&b1_full[k % S1], (k / S1) & 1, a.err);
        for (uint32_t k = it > S2 ? it - S2 : 0; k < it; ++k) mbar_wait(&b2_full[k % S2], (k / S2) & 1, a.err);
        if (items) mbar_wait(&a_full, (items - 1) & 1, a.err);
      }
    } else if (warp == 1) {
      // ---- MMA issuer
      constexpr uint32_t id_x = umma_idesc_bf16(kAttnRows, kAttnRows), id_acc = umma_idesc_bf16_bmn(kAttnRows, HD);
      uint32_t it = 0, items = 0;
      const uint32_t tmem = uniform(s_tmem);
      BwdItem t;
      auto b1 = [&](uint32_t k) { return base + SM::kB1 + (k % S1) * SM::kTile; };
      auto b2 = [&](uint32_t k) { return base + SM::kB2 + (k % S2) * SM::kTile; };
      auto product_x = [&](uint32_t k) {  // streamed block k (counted over all items)
        wait(&b1_full[k % S1], (k / S1) & 1);
        tc_fence_after();
        const uint32_t buf = kTwoX ? k & 1 : 0;
        attn_mma_ss<HD>(tmem + tX + 128 * buf, base + SM::kA, b1(k), id_x);
        umma_commit_warp(&x_full[buf]);
      };
      auto product_y = [&](uint32_t k) {
        wait(&b2_full[k % S2], (k / S2) & 1);
        tc_fence_after();
        attn_mma_ss<HD>(tmem + tY, base + SM::kA + SM::kTile, b2(k), id_x);
        umma_commit_warp(&y_full);
      };
      while (next_item(t)) {
        t.n = (int)uniform(t.n);
        if (t.n == 0) continue;
        wait(&a_full, items & 1);
        tc_fence_after();
        product_x(it);
        product_y(it);
        if constexpr (!KV) umma_commit_warp(&b2_empty[it % S2]);
        if (kAhead && t.n > 1) product_x(it + 1);
        if (t.n == 1) umma_commit_warp(&a_empty);
        for (int i = 0; i < t.n; ++i, ++it) {
          const bool more = i + 1 < t.n;
          const uint32_t x = tmem + tX + (kTwoX ? 128 * (it & 1) : 0);
          if constexpr (KV) {
            wait(&p_full, it & 1);
            if (i == 0 && items > 0) wait(&acc_free, (items - 1) & 1);
            tc_fence_after();
            attn_mma_ts(tmem + tAcc1, x, 64, b2(it), id_acc, i > 0);
            umma_commit_warp(&b2_empty[it % S2]);
            if (!kTwoX && more) product_x(it + 1);
            wait(&ds_full, it & 1);
            tc_fence_after();
            if (kTwoX && more) product_y(it + 1);  // Y has been read: it need not wait behind dS Q
            attn_mma_ts(tmem + tAcc2, kTwoX ? x + kDsOff : tmem + tY, 64, b1(it), id_acc, i > 0);
            umma_commit_warp(&b1_empty[it % S1]);
            if (!kTwoX && more) product_y(it + 1);
          } else {
            if (!kAhead && more) product_x(it + 1);
            wait(&ds_full, it & 1);
            if (more) {
              product_y(it + 1);
              umma_commit_warp(&b2_empty[(it + 1) % S2]);
            }
            if (i == 0 && items > 0) wait(&acc_free, (items - 1) & 1);
            tc_fence_after();
            attn_mma_ts(tmem + tAcc1, x, 64, b1(it), id_acc, i > 0);
            umma_commit_warp(&b1_empty[it % S1]);
          }
          if (kAhead && i + 2 < t.n) product_x(it + 2);
          if (i + 2 == t.n) umma_commit_warp(&a_empty);  // the last X and Y are issued
        }
        umma_commit_warp(&acc_done);
        ++items;
      }
      umma_commit_warp(&mma_done);  // nothing it issued may still run when the CTA exits
      if (lane == 0) mbar_wait(&mma_done, 0, a.err);
    } else if (warp == 2) {
      // ---- finder
      // A key/value item has all query heads of its part, whether a tile holds one or several.
      const uint32_t units = KV ? (SPLIT ? a.n_kv * a.splits : a.n_kv) : a.n_q;
      const bool several = a.group > (SPLIT ? a.splits : 1);
      AttnOrder ord{a.cu,
                    a.batch,
                    kAttnRows,
                    units,
                    several ? (KV ? units : (uint32_t)(a.n_kv * ((a.group + 1) / 2))) : 0u,
                    several ? (KV ? units : (uint32_t)(a.n_kv * ((a.group + 3) / 4))) : 0u,
                    s_cache};
      const bool ok = ord.init(a.T, lane);
      if (!ok && blockIdx.x == 0 && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDevBadSequence);
      const uint32_t work = ord.work();  // below 2^31: the host checks
      for (uint32_t k = 0;; ++k) {
        const uint32_t s = k % kBwdSched;
        if (!__all_sync(0xffffffffu, wait(&it_empty[s], ((k / kBwdSched) & 1) ^ 1))) break;
        const uint32_t w = attn_deal(k, blockIdx.x, gridDim.x);
        BwdItem t = {};
        t.valid = k * gridDim.x < work;  // else no CTA has any left
        if (w < work) {                  // (an empty item: this CTA has none in the last round)
          int seq, cost;
          ord.find(w, lane, seq, cost, t.head, t.hs);
          const int heads = SPLIT ? a.group / a.splits : a.group, fit = 4 >> t.hs;  // heads that fit a tile
          const int tiles = (heads + fit - 1) >> (2 - t.hs);
          if constexpr (KV) {
            t.split = t.head / a.n_kv;
            t.head -= t.split * a.n_kv;
            t.end = t.head * a.group + (t.split + 1) * heads;
          } else {
            const int kvh = t.head / (t.hs == 2 ? a.group : tiles);
            if (t.hs != 2) t.head = kvh * a.group + (t.head - kvh * tiles) * fit;
            t.end = (kvh + 1) * a.group;
          }
          t.first = a.cu[seq];
          t.len = a.cu[seq + 1] - t.first;
          t.blk = KV ? (t.len + kAttnRows - 1) / kAttnRows - cost : cost - 1;
          t.own = t.first + kAttnRows * t.blk;
          t.n = KV ? cost * tiles : cost;
        }
        if (lane == 0) {
          s_item[s] = t;
          mbar_arrive(&it_full[s]);
        }
        __syncwarp();
        if (!t.valid) break;
      }
    } else if (warp == 3) {
      if constexpr (KV) {
        // ---- lse and delta of the streamed rows; a row behind the end gets p = 2^(x - inf) = 0
        uint32_t it = 0;
        BwdItem t;
        while (next_item(t)) {
          for (int i = 0; i < t.n; ++i, ++it) {
            int head;
            const int blk = block_of(t, i, head);
            const uint32_t s = it % kStatStages;
            float ls[4], de[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = kAttnRows * blk + 32 * (x & ((1 << t.hs) - 1)) + lane;
              const bool in = r < t.len && head + (x >> t.hs) < t.end;
              const int64_t at = (int64_t)(head + (x >> t.hs)) * a.T + t.first + r;
              ls[x] = in ? -a.lse[at] * kLog2e : -INFINITY;
              de[x] = in ? -a.delta[at] : 0.f;
              if (ls[x] == INFINITY) ls[x] = -INFINITY;  // a row without keys
            }
            if (it >= kStatStages) wait(&st_empty[s], ((it / kStatStages) - 1) & 1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              s_stat[s][0][32 * x + lane] = ls[x];
              s_stat[s][1][32 * x + lane] = de[x];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&st_full[s]);
          }
        }
      } else if (a.zero_rest) {
        bool none = a.batch == 0;
        for (int s = lane; s < a.batch; s += 32) none |= a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.T;
        none = __any_sync(0xffffffffu, none);
        const int64_t first = none ? 0 : a.cu[0], last = none ? 0 : a.cu[a.batch];
        attn_zero_rows(a.dq, a.T, a.n_q * (HD / 8), first, last, lane);
        attn_zero_rows(a.dk, a.T, a.n_kv * (HD / 8), first, last, lane);
        attn_zero_rows(a.dv, a.T, a.n_kv * (HD / 8), first, last, lane);
      }
    }
  } else {
    regs_more<208>();
    // ---- P and dS, and the results
    const int wg = (warp - 4) >> 2, qtr = warp & 3, row = 32 * qtr + lane;
    const uint32_t lanes = (uint32_t)(32 * qtr) << 16;
    const float c = a.scale_log2;
    uint32_t it = 0, items = 0;
    BwdItem t;
    while (next_item(t)) {
      if (t.n == 0) continue;
      float r_lse = 0.f, r_delta = 0.f;  // query kernel: -lse log2(e) and -delta of this row
      // query kernel: the head and the row in the block that this thread's row is
      const int q_head = t.head + (KV ? 0 : qtr >> t.hs), q_row = KV ? row : 32 * (qtr & ((1 << t.hs) - 1)) + lane;
      const bool in = kAttnRows * t.blk + q_row < t.len && (KV || q_head < t.end);
      if constexpr (!KV) {
        const int64_t at = (int64_t)q_head * a.T + t.own + q_row;
        r_lse = in ? -a.lse[at] * kLog2e : -INFINITY;
        if (r_lse == INFINITY) r_lse = -INFINITY;
        if (t.n > 1) {  // delta = dout . out: half a row's columns each, dout from the CTA's own tile
          constexpr int CH = HD / 16;
          const uint4* src = a.out + ((int64_t)(t.own + row) * a.n_q + t.head) * (HD / 8) + CH * wg;
          const unsigned char* tile = base + SM::kA + SM::kTile + (HD / 64 - 1) * wg * kAttnBox;
          uint4 w[CH];
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) w[ch] = in ? src[ch] : make_uint4(0, 0, 0, 0);
          wait(&a_full, items & 1);
          float s = 0.f;
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            float x[8], y[8];
            unpack8(w[ch], x);
            unpack8(*reinterpret_cast<const uint4*>(tile + attn_swz(row, (HD == 64 ? CH * wg : 0) + ch)), y);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
          }
          s_stat[wg][0][row] = s;
          named_sync(1, 256);  // (nobody writes there again before every warp's dS of this item)
          r_delta = -(s_stat[0][0][row] + s_stat[1][0][row]);
          if (wg == 0 && in) a.delta[at] = -r_delta;
        }
      }
      const uint64_t c2 = pair(c, c);
#pragma unroll 1
      for (int i = 0; i < t.n; ++i, ++it) {
        int head;
        const bool diagonal = block_of(t, i, head) == t.blk;
        const uint32_t buf = kTwoX ? it & 1 : 0;
        const uint32_t t_x = tmem + lanes + tX + 128 * buf + 64 * wg, t_y = tmem + lanes + tY + 64 * wg;
        const float* st = s_stat[KV ? it % kStatStages : 0][0] + 64 * wg;
        uint64_t ls2[KV ? 32 : 1];
        if constexpr (KV) {  // before X is here
          wait(&st_full[it % kStatStages], (it / kStatStages) & 1);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(st + 2 * e);
            ls2[e] = v.x;
            ls2[e + 1] = v.y;
          }
        } else {
          ls2[0] = pair(r_lse, r_lse);
        }
        wait(&x_full[buf], kTwoX ? (it >> 1) & 1 : it & 1);
        tc_fence_after();
        float p[64], y[64];
        tmem_ld64(t_x, p);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float &p0 = p[32 * x + 2 * e], &p1 = p[32 * x + 2 * e + 1];
            unpair(fma2(pair(p0, p1), c2, ls2[KV ? 16 * x + e : 0]), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
          }
          if constexpr (KV) {
            const int piece = (2 * wg + x) & ((1 << t.hs) - 1);
            if (diagonal && piece <= qtr) {  // queries before this key do not attend it
              asm volatile("");              // a branch, not selects in every block
              const int first = piece < qtr ? 32 : lane;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < first) p[32 * x + e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2(p[32 * x + 2 * e], p[32 * x + 2 * e + 1]);
            tmem_st16(t_x + 16 * x, w);
          }
        }
        if constexpr (KV) {
          tmem_wait_st();
          tc_fence_before();
          // Where X has two buffers, nothing else keeps a warp from P of this block while the
          // issuer has yet to see p_full of the block before (or another warp to arrive
          // there). P dO of the block before, issued after that, frees its streamed tile.
          if (kTwoX && it > 0) wait(&b2_empty[(it - 1) % S2], ((it - 1) / S2) & 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full);
        }
        wait(&y_full, it & 1);
        tc_fence_after();
        tmem_ld64(t_y, y);
        if constexpr (!KV) {
          if (diagonal) {  // keys after the row (and so behind the sequence), whatever was computed there
            asm volatile("");
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (64 * wg + e > q_row) p[e] = y[e] = 0.f;
          }
          if (t.n == 1) {
            // Rows with few keys: delta = sum_j p_ij dp_ij is summed here, from the p and
            // dp that it is subtracted from. dout . out with out rounded to bf16 is off
            // by up to 2^-8 of |dout| |out|, which a sharp row of few keys, whose ds are small
            // differences, would feel; in later blocks it is lost among the others.
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              s0 += p[e];
              s1 = fmaf(p[e], y[e], s1);
            }
            s_stat[wg][0][row] = s0;
            s_stat[wg][1][row] = s1;
            named_sync(1, 256);
            r_delta = -(s_stat[0][1][row] + s_stat[1][1][row]) / (s_stat[0][0][row] + s_stat[1][0][row]);
            if (wg == 0 && in) a.delta[(int64_t)q_head * a.T + t.own + q_row] = -r_delta;
          }
        }
        const uint32_t t_ds = KV && !kTwoX ? t_y : t_x + kDsOff;
        const uint64_t d2 = pair(r_delta, r_delta);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            uint64_t n0 = d2, n1 = d2;  // -delta of two pairs of columns
            if constexpr (KV) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(st + kAttnRows + 32 * x + 2 * e);
              n0 = v.x;
              n1 = v.y;
            }
            const int k = 32 * x + 2 * e;
            float a0, a1, b0, b1;
            unpair(mul2(pair(p[k], p[k + 1]), add2(pair(y[k], y[k + 1]), n0)), a0, a1);
            unpair(mul2(pair(p[k + 2], p[k + 3]), add2(pair(y[k + 2], y[k + 3]), n1)), b0, b1);
            w[e] = pack2(a0, a1);
            w[e + 1] = pack2(b0, b1);
          }
          tmem_st16(t_ds + 16 * x, w);
        }
        if constexpr (KV) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&st_empty[it % kStatStages]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full);
      }
      wait(&acc_done, items & 1);
      ++items;
      tc_fence_after();
      // key/value kernel: warps 4-7 store dv, 8-11 dk; query kernel: each half of dq's columns
      constexpr int COLS = KV ? HD : HD / 2, UNIT = 32;
      const uint32_t t_acc = tmem + lanes + (KV ? (wg ? tAcc2 : tAcc1) : tAcc1 + COLS * wg);
      float o[COLS];
#pragma unroll
      for (int x = 0; x < COLS / 32; ++x) tmem_ld32(t_acc + 32 * x, o + 32 * x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_free);
      const float f = KV && wg == 0 ? 1.f : a.scale;
      uint4* out = KV ? (wg ? a.dk : a.dv) : a.dq;
      const int heads = KV ? a.n_kv : a.n_q, col0 = KV ? 0 : COLS * wg;
      const int row0 = t.own + q_row - lane, rows = KV || q_head < t.end ? t.first + t.len - row0 : 0;
      if constexpr (SPLIT) {  // sums over this part of the group, for the folding kernel
        if (lane < rows) {
          float4* dst = reinterpret_cast<float4*>(
              a.part + (((2 * t.split + wg) * a.T + row0 + lane) * (int64_t)a.n_kv + q_head) * HD);
#pragma unroll
          for (int e = 0; e < COLS / 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      } else if constexpr (HD == 128) {
        uint4* dst = out + ((int64_t)(row0 + lane) * heads + q_head) * (HD / 8) + col0 / 8;
        if (lane < rows)
#pragma unroll
          for (int ch = 0; ch < COLS / 8; ++ch) {
            const float* v = o + 8 * ch;
            dst[ch] = make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f),
                                 pack2(v[6] * f, v[7] * f));
          }
      } else if (rows > 0) {
        unsigned char* sbuf = base + SM::kOut + (warp - 4) * kStageBytes;
        constexpr int CHU = UNIT / 8, RP = 32 / CHU;  // chunks per staged row, rows per pass
        auto at = [](int r, int ch) { return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4); };  // no bank conflicts either way
#pragma unroll
        for (int x = 0; x < COLS / UNIT; ++x) {
#pragma unroll
          for (int ch = 0; ch < CHU; ++ch) {
            const float* v = o + UNIT * x + 8 * ch;
            *reinterpret_cast<uint4*>(sbuf + at(lane, ch)) =
                make_uint4(pack2(v[0] * f, v[1] * f), pack2(v[2] * f, v[3] * f), pack2(v[4] * f, v[5] * f),
                           pack2(v[6] * f, v[7] * f));
          }
          __syncwarp();
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += RP) {
            const int r = r0 + lane / CHU, ch = lane % CHU;
            const uint4 v = *reinterpret_cast<const uint4*>(sbuf + at(r, ch));
            if (r < rows) out[((int64_t)(row0 + r) * heads + q_head) * (HD / 8) + (col0 + UNIT * x) / 8 + ch] = v;
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  attn_report(&s_watch, a.err);
}

// dv and dk from the parts of each group's query heads, in their order. Rows of the
// sequences only.
__global__ void __launch_bounds__(256) qkvp_attention_fold_kernel(const AttnBwdArgs a, int row4) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = a.batch == 0;
  __syncthreads();
  for (int s = threadIdx.x; s < a.batch; s += 256)
    if (a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.T) s_bad = 1;
  __syncthreads();
  if (s_bad) return;
  const int64_t first = (int64_t)a.cu[0] * row4, n = (int64_t)a.cu[a.batch] * row4 - first, all = a.T * row4;
  const float4* part = reinterpret_cast<const float4*>(a.part);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * n; i += (int64_t)gridDim.x * 256) {
    const bool dk = i >= n;
    const int64_t at = first + (dk ? i - n : i);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < a.splits; ++k) {
      const float4 x = part[(2 * k + dk) * all + at];
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
    const float f = dk ? a.scale : 1.f;
    reinterpret_cast<uint2*>(dk ? a.dk : a.dv)[at] = make_uint2(pack2(v.x * f, v.y * f), pack2(v.z * f, v.w * f));
  }
}

const void* attention_fold_kernel() { return reinterpret_cast<const void*>(&qkvp_attention_fold_kernel); }

template <int HD>
static const void* bwd_kernel(bool kv, bool split) {
  if (!kv) return reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<HD, false, false>);
  return split ? reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<HD, true, true>)
               : reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<HD, true, false>);
}
const void* attention_bwd_kernel(int head_dim, bool kv, bool split) {
  return head_dim == 64 ? bwd_kernel<64>(kv, split) : bwd_kernel<128>(kv, split);
}
int attention_bwd_smem_bytes(int head_dim) {
  return head_dim == 64 ? BwdSmem<64>::kBytes : BwdSmem<128>::kBytes;
}
int attention_bwd_threads() { return kBwdThreads; }

}  // namespace qkvp
