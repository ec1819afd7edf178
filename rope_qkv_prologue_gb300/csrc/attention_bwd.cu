// Backward of the causal attention over packed sequences (sm_103a): dq, dk and
// dv from dout, the inputs and the forward's out and lse.
//
// With p_ij = e^(s_ij - lse_i), delta_i = dout_i . out_i, dp_ij = dout_i . v_j and
// ds_ij = p_ij (dp_ij - delta_i):
//     dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j,
// dk and dv summed over the query heads of the group too. Three kernels:
//   1. qkvp_attention_delta_kernel: delta, one pass over dout and out;
//   2. the key/value kernel: a CTA owns 128 keys of one key/value head and goes
//      through the query blocks and heads that attend them, forming the transposed
//      S^T = K Q^T and dP^T = V dO^T and adding P^T dO and dS^T Q;
//   3. the query kernel: a CTA owns 128 queries of one head and goes through its
//      keys, adding dS K.
// S and dP are formed twice (seven products instead of five), so that every result
// is a sum in one CTA's tensor memory in a fixed order: no atomics, no partial
// results in memory, the same bits every time.
//
// Both kernels are one template: two tiles of the CTA's own rows stay in shared
// memory, pairs of tiles stream past them by TMA, X = A1 B1^T and Y = A2 B2^T go
// to tensor memory, 256 threads turn them into bf16 P and dS in tensor memory (in
// the columns they came from), and those are the first operands of the
// accumulating products. A thread owns a row and half of a block's columns. MMAs
// execute in order, so the next X may be issued over the P that the product before
// it reads; the order (key/value kernel)
//     P dO (i), X (i + 1), dS Q (i), Y (i + 1), ...
// keeps the tensor cores on one pair of products while the threads work on the
// other. P and dS are rounded to bf16 as operands; all sums are fp32.
//   warp 0      loads tiles (and zeroes rows behind a sequence's end in those that
//               are summed over: 0 times whatever is there need not be 0);
//   warp 1      issues the MMAs;
//   warp 2      finds work items (AttnOrder), one ahead;
//   warp 3      key/value kernel: lse and delta of the streamed rows;
//   warps 4-11  the arithmetic between the products, and the results' stores.
#include "attention.cuh"

namespace qkvp {
namespace {

constexpr int kBwdThreads = 384;
constexpr int kBwdSched = 2;
constexpr int kStatStages = 2;
constexpr int kStageBytes = 32 * 64;  // a warp's store buffer: 32 rows x 32 bf16

template <int HD>
struct BwdSmem {
  static constexpr int kTile = (HD / 64) * kAttnBox;
  static constexpr int kStages = HD == 128 ? 2 : 4;  // of each streamed operand
  static constexpr int kA = 0;
  static constexpr int kB1 = 2 * kTile;
  static constexpr int kB2 = kB1 + kStages * kTile;
  static constexpr int kOut = kB2 + kStages * kTile;
  static constexpr int kBytes = kOut + 8 * kStageBytes;
};

struct BwdItem {
  int n;      // streamed blocks
  int own;    // first row of the CTA's own block, of T
  int first;  // first row of the sequence
  int len;    // its rows
  int blk;    // the own block's index in the sequence
  int head;   // key/value head, or query head
  int valid;
};

}  // namespace

template <int HD, bool KV>
__global__ void __launch_bounds__(kBwdThreads, 1)
    qkvp_attention_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                              const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                              const AttnBwdArgs a) {
  using SM = BwdSmem<HD>;
  constexpr int ST = SM::kStages;
  constexpr uint32_t tX = 0, tY = KV ? 128 : 256, tAcc1 = KV ? 256 : 384, tAcc2 = KV ? 256 + HD : 384;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t a_full, a_empty, b1_full[ST], b1_empty[ST], b2_full[ST], b2_empty[ST], tail_bar,
      x_full[2], y_full, p_full, ds_full, acc_done, acc_free, st_full[kStatStages], st_empty[kStatStages],
      it_full[kBwdSched], it_empty[kBwdSched], mma_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  __shared__ BwdItem s_item[kBwdSched];
  __shared__ int s_cache[AttnOrder::kCached];
  __shared__ __align__(16) float s_stat[KV ? kStatStages : 1][2][kAttnRows];  // lse log2(e), delta
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&a_full, 1);
    mbar_init(&a_empty, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&b1_full[s], 1);
      mbar_init(&b1_empty[s], 1);
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
    s_fail = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(&s_tmem, 512);
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* fail = &s_fail;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = attn_wait(bar, parity, fail);
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
      const int per = t.n / a.group;
      head = t.head * a.group + i / per;
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
      if (lane == 0) {
        mbar_arrive_expect_tx(&a_full, 2 * SM::kTile);
        for (int x = 0; x < HD / 64; ++x) {
          tma_load_2d(base + SM::kA + x * kAttnBox, KV ? &tmap_k : &tmap_q, t.head * HD + 64 * x, t.own, &a_full);
          tma_load_2d(base + SM::kA + SM::kTile + x * kAttnBox, KV ? &tmap_v : &tmap_do, t.head * HD + 64 * x, t.own,
                      &a_full);
        }
      }
      for (int i = 0; i < t.n; ++i, ++it) {
        int head;
        const int blk = block_of(t, i, head);
        const uint32_t s = it % ST;
        const int rows = t.len - kAttnRows * blk;  // of the sequence in this block
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint64_t* full = which ? &b2_full[s] : &b1_full[s];
          if (it >= ST) wait(which ? &b2_empty[s] : &b1_empty[s], ((it / ST) - 1) & 1);
          unsigned char* dst = base + (which ? SM::kB2 : SM::kB1) + s * SM::kTile;
          const CUtensorMap* map = KV ? (which ? &tmap_do : &tmap_q) : (which ? &tmap_v : &tmap_k);
          const bool patch = rows < kAttnRows && (KV || which == 0);
          uint64_t* bar = patch ? &tail_bar : full;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, SM::kTile);
            for (int x = 0; x < HD / 64; ++x)
              tma_load_2d(dst + x * kAttnBox, map, head * HD + 64 * x, t.first + kAttnRows * blk, bar);
          }
          if (patch) {
            wait(&tail_bar, tails++ & 1);
            for (int r = rows + (lane >> 3); r < kAttnRows; r += 4)
              for (int x = 0; x < HD / 64; ++x)
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
      for (uint32_t k = it > ST ? it - ST : 0; k < it; ++k) {
        mbar_wait(&b1_full[k % ST], (k / ST) & 1, a.err);
        mbar_wait(&b2_full[k % ST], (k / ST) & 1, a.err);
      }
      if (items) mbar_wait(&a_full, (items - 1) & 1, a.err);
    }
  } else if (warp == 1) {
    // ---- MMA issuer
    constexpr uint32_t id_x = umma_idesc_bf16(kAttnRows, kAttnRows), id_acc = umma_idesc_bf16_bmn(kAttnRows, HD);
    uint32_t it = 0, items = 0;
    const uint32_t tmem = uniform(s_tmem);
    BwdItem t;
    auto b1 = [&](uint32_t k) { return base + SM::kB1 + (k % ST) * SM::kTile; };
    auto b2 = [&](uint32_t k) { return base + SM::kB2 + (k % ST) * SM::kTile; };
    auto product_x = [&](uint32_t k) {  // streamed block k (counted over all items)
      wait(&b1_full[k % ST], (k / ST) & 1);
      tc_fence_after();
      const uint32_t buf = KV ? 0 : k & 1;
      attn_mma_ss<HD>(tmem + tX + 128 * buf, base + SM::kA, b1(k), id_x);
      umma_commit_warp(&x_full[buf]);
    };
    auto product_y = [&](uint32_t k) {
      wait(&b2_full[k % ST], (k / ST) & 1);
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
      if constexpr (!KV) umma_commit_warp(&b2_empty[it % ST]);
      if (t.n == 1) umma_commit_warp(&a_empty);
      for (int i = 0; i < t.n; ++i, ++it) {
        const bool more = i + 1 < t.n;
        if constexpr (KV) {
          wait(&p_full, it & 1);
          if (i == 0 && items > 0) wait(&acc_free, (items - 1) & 1);
          tc_fence_after();
          attn_mma_ts(tmem + tAcc1, tmem + tX, 64, b2(it), id_acc, i > 0);
          umma_commit_warp(&b2_empty[it % ST]);
          if (more) product_x(it + 1);
          wait(&ds_full, it & 1);
          tc_fence_after();
          attn_mma_ts(tmem + tAcc2, tmem + tY, 64, b1(it), id_acc, i > 0);
          umma_commit_warp(&b1_empty[it % ST]);
          if (more) product_y(it + 1);
        } else {
          if (more) product_x(it + 1);
          wait(&ds_full, it & 1);
          if (i == 0 && items > 0) wait(&acc_free, (items - 1) & 1);
          tc_fence_after();
          attn_mma_ts(tmem + tAcc1, tmem + tX + 128 * (it & 1), 64, b1(it), id_acc, i > 0);
          umma_commit_warp(&b1_empty[it % ST]);
          if (more) {
            product_y(it + 1);
            umma_commit_warp(&b2_empty[(it + 1) % ST]);
          }
        }
        if (i + 2 == t.n) umma_commit_warp(&a_empty);  // the last X and Y are issued
      }
      umma_commit_warp(&acc_done);
      ++items;
    }
    umma_commit_warp(&mma_done);  // nothing it issued may still run when the CTA exits
    if (lane == 0) mbar_wait(&mma_done, 0, a.err);
  } else if (warp == 2) {
    // ---- finder
    AttnOrder ord{a.cu, a.batch, kAttnRows, s_cache, 0, 0};
    const bool ok = ord.init(a.T, lane);
    if (!ok && blockIdx.x == 0 && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDevBadSequence);
    const int units = KV ? a.n_kv : a.n_q;
    const uint32_t work = ord.total * (uint32_t)units;  // below 2^31: the host checks
    for (uint32_t k = 0;; ++k) {
      const uint32_t s = k % kBwdSched;
      if (!__all_sync(0xffffffffu, wait(&it_empty[s], ((k / kBwdSched) & 1) ^ 1))) break;
      const uint32_t w = attn_deal(k, blockIdx.x, gridDim.x);
      BwdItem t = {};
      t.valid = k * gridDim.x < work;  // else no CTA has any left
      if (w < work) {                  // (an empty item: this CTA has none in the last round)
        int seq, cost;
        const uint32_t rank = w / (uint32_t)units;
        ord.find(rank, lane, seq, cost);
        t.head = (int)(w - rank * (uint32_t)units);
        t.first = a.cu[seq];
        t.len = a.cu[seq + 1] - t.first;
        t.blk = KV ? (t.len + kAttnRows - 1) / kAttnRows - cost : cost - 1;
        t.own = t.first + kAttnRows * t.blk;
        t.n = KV ? cost * a.group : cost;
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
            const int r = kAttnRows * blk + 32 * x + lane;
            const bool in = r < t.len;
            const int64_t at = (int64_t)head * a.T + t.first + r;
            ls[x] = in ? a.lse[at] * kLog2e : INFINITY;
            de[x] = in ? a.delta[at] : 0.f;
            if (ls[x] == -INFINITY) ls[x] = INFINITY;
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
      float r_lse = 0.f, r_delta = 0.f;
      if constexpr (!KV) {
        const int64_t at = (int64_t)t.head * a.T + t.own + row;
        const bool in = kAttnRows * t.blk + row < t.len;
        r_lse = in ? a.lse[at] * kLog2e : INFINITY;
        r_delta = in ? a.delta[at] : 0.f;
        if (r_lse == -INFINITY) r_lse = INFINITY;
      }
      for (int i = 0; i < t.n; ++i, ++it) {
        int head;
        const bool diagonal = block_of(t, i, head) == t.blk;
        const uint32_t buf = KV ? 0 : it & 1;
        const uint32_t t_x = tmem + lanes + tX + 128 * buf + 64 * wg, t_y = tmem + lanes + tY + 64 * wg;
        wait(&x_full[buf], KV ? it & 1 : (it >> 1) & 1);
        tc_fence_after();
        float p[64];
        tmem_ld32(t_x, p);
        tmem_ld32(t_x + 32, p + 32);
        const float* st = s_stat[KV ? it % kStatStages : 0][0] + 64 * wg;
        if constexpr (KV) {
          wait(&st_full[it % kStatStages], (it / kStatStages) & 1);
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(st + e);
            p[e] = ex2(fmaf(p[e], c, -v.x));
            p[e + 1] = ex2(fmaf(p[e + 1], c, -v.y));
            p[e + 2] = ex2(fmaf(p[e + 2], c, -v.z));
            p[e + 3] = ex2(fmaf(p[e + 3], c, -v.w));
          }
          if (diagonal)  // queries before this key do not attend it
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (64 * wg + e < row) p[e] = 0.f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2(p[32 * x + 2 * e], p[32 * x + 2 * e + 1]);
            tmem_st16(t_x + 16 * x, w);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full);
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) p[e] = ex2(fmaf(p[e], c, -r_lse));
        }
        wait(&y_full, it & 1);
        tc_fence_after();
        float y[64];
        tmem_ld32(t_y, y);
        tmem_ld32(t_y + 32, y + 32);
        if constexpr (KV) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(st + kAttnRows + e);
            p[e] *= y[e] - v.x;
            p[e + 1] *= y[e + 1] - v.y;
            p[e + 2] *= y[e + 2] - v.z;
            p[e + 3] *= y[e + 3] - v.w;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&st_empty[it % kStatStages]);
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) p[e] *= y[e] - r_delta;
          if (diagonal)  // keys after the row (and so behind the sequence), whatever was computed there
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (64 * wg + e > row) p[e] = 0.f;
        }
        const uint32_t t_ds = KV ? t_y : t_x;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack2(p[32 * x + 2 * e], p[32 * x + 2 * e + 1]);
          tmem_st16(t_ds + 16 * x, w);
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
      unsigned char* sbuf = base + SM::kOut + (warp - 4) * kStageBytes;
      const int row0 = t.own + 32 * qtr, rows = t.first + t.len - row0;
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
          if (r < rows) out[((int64_t)(row0 + r) * heads + t.head) * (HD / 8) + (col0 + UNIT * x) / 8 + ch] = v;
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  attn_report(fail, a.err);
}

// delta[h, t] = dout[t, h] . out[t, h] in fp32, and (where asked for) zeros in the
// gradients' rows of no sequence. Bound by reading dout and out once.
template <int HD>
__global__ void __launch_bounds__(256) qkvp_attention_delta_kernel(const AttnBwdArgs a) {
  constexpr int L = HD / 8, RW = 32 / L;  // lanes per row, rows per warp
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n = a.T * a.n_q;
  const int64_t step = (int64_t)gridDim.x * 8 * RW;
  for (int64_t r0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * RW; r0 < n; r0 += step) {
    const int64_t r = r0 + lane / L;
    float s = 0.f;
    if (r < n) {
      float x[8], y[8];
      unpack8(a.out[r * L + lane % L], x);
      unpack8(a.dout[r * L + lane % L], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane % L == 0 && r < n) a.delta[(r % a.n_q) * a.T + r / a.n_q] = s;
  }
  if (a.zero_rest && threadIdx.x < 32) {
    bool bad = false;
    for (int s = lane; s < a.batch; s += 32) bad |= a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.T;
    bad = __any_sync(0xffffffffu, bad) || a.batch == 0;
    const int64_t first = bad ? 0 : a.cu[0], last = bad ? 0 : a.cu[a.batch];
    attn_zero_rows(a.dq, a.T, a.n_q * L, first, last, lane);
    attn_zero_rows(a.dk, a.T, a.n_kv * L, first, last, lane);
    attn_zero_rows(a.dv, a.T, a.n_kv * L, first, last, lane);
  }
}

const void* attention_bwd_kernel(int head_dim, bool kv) {
  if (head_dim == 64)
    return kv ? reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<64, true>)
              : reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<64, false>);
  return kv ? reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<128, true>)
            : reinterpret_cast<const void*>(&qkvp_attention_bwd_kernel<128, false>);
}
const void* attention_delta_kernel(int head_dim) {
  return head_dim == 64 ? reinterpret_cast<const void*>(&qkvp_attention_delta_kernel<64>)
                        : reinterpret_cast<const void*>(&qkvp_attention_delta_kernel<128>);
}
int attention_bwd_smem_bytes(int head_dim) {
  return (head_dim == 64 ? BwdSmem<64>::kBytes : BwdSmem<128>::kBytes) + 1024;
}
int attention_bwd_threads() { return kBwdThreads; }

}  // namespace qkvp
