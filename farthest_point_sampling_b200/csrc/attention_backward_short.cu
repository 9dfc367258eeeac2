// Attention of packed events, backward, for events of at most 128 queries and
// 128 keys (the tokenizer's usual K): all three gradients in one kernel.
//
// Such an event is one tile, so S and dP are formed once,
//   S^T = K Q^T,  dP^T = V dO^T,  P = exp2(c S - lse),  dS = P (dP - D),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K,
// and q, k, v, out and dout are read once and the gradients written once: with
// 64-wide heads and 128 tokens that traffic, 8 tensors of it, bounds the
// kernel, not the products.  2048 events of up to 128 tokens, 12 heads of 64:
// 742 us, 3.7 TB/s; the same events through the kernels of attention_backward.cu
// took 982.  What is left is latency: a unit's phases wait for one another.
//
// A work item is an event and a key head, with a unit for each query head of
// its group; dK and dV are summed over the units in TMEM.  Warps: a loading
// and an issuing warp, and eight for the rest with two threads per key row,
// each for half of the queries.  P goes back over S in TMEM as 16-bit operand
// A; dS goes to shared memory, where it is read along its rows for dK and
// across them for dQ.
//
// The phases of a unit (scores, weights, gradients, stores) follow one another,
// so what fills an SM is a second block: with 64-wide heads of their own keys
// (kTwo) a block makes do with 256 columns of TMEM, dK and dQ in the place of dP
// and dV in that of the scores that P does not cover (the same events with one
// block an SM took 923 us).  Otherwise one block takes the SM, with dV and dK kept
// over the heads of a group.  The two 32-query chunks of a thread go through one
// loop body, which keeps the kernel in the instruction cache and a thread at 96
// registers.
//
// Rounding: as in attention_backward.cu.
#include <type_traits>

#include "attention_plan.h"
#include "attention_short.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace fpstok {

namespace {

constexpr int kHalf = kTile / 2;
constexpr int kPanel = kTile * 128;
constexpr int kSoftmaxThreads = 256;
constexpr int kShortThreads = kSoftmaxThreads + 64;
constexpr int kItemRing = 2;
constexpr uint32_t kColS = 0, kColDP = 128;

struct ShortArgs {
  int64_t n_q, n_kv;
  int heads, kv_heads, group, D;
  AttnMask mask;
  float scale, scale_log2;
  const void* out;
  const float* lse;
  const float* rows;  // [2][heads, n_q]: the second half holds -D of queries that see few keys
  const float* range;  // float16: see attention_backward_range.cu
  void *dq, *dk, *dv;
  const int64_t *q_offsets, *kv_offsets;
  int B;
  WaitTest test;
  bool sectors;  // every gradient row starts on a 32-byte sector, and ends on one
  const TileItem* items;
  WsHeader* hdr;
};

// One work item as the loading warp hands it to the others; nq = -1 ends the work.
template <bool kScaled>
struct ShortItem : ItemScale<kScaled> {
  int h, q_row, nq, k_row, nk;  // key head; the event's first query and key rows, queries, keys
};

template <int DP, bool kTwo>
struct ShortShape {
  static constexpr int kPanels = DP / 64;
  static constexpr uint32_t kTileBytes = kPanels * kPanel;
  static constexpr int kStages = DP == 64 && !kTwo ? 2 : 1;  // of (K, V), and of (Q, dO)
  static constexpr uint32_t kColumns = kTwo ? 256 : 512;
  // 64-wide heads leave room for dQ beside dV and dK; with 128-wide ones it takes the place of dP
  static constexpr uint32_t kColDV = 256, kColDK = kTwo ? kColDP : 256 + DP;
  static constexpr uint32_t kColDQ = kTwo ? kColDP + 64 : DP == 64 ? kColDK + DP : kColDP;
  static constexpr size_t kSmem = 1024 + 4 * kStages * kTileBytes + 2 * kPanel + 2 * kTile * sizeof(float) +
                                  kItemRing * sizeof(ShortItem<true>) + 512;
};

template <typename T, int DP, bool kTwo>
__global__ void __launch_bounds__(kShortThreads, kTwo ? 2 : 1)
    k_attn_backward_short(const ShortArgs a, const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const __grid_constant__ CUtensorMap map_do) {
  using Sh = ShortShape<DP, kTwo>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kStages = Sh::kStages;
  constexpr int kLoadWarp = kSoftmaxThreads / 32, kMmaWarp = kLoadWarp + 1;
  extern __shared__ uint8_t s_raw[];
  uint8_t* s_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* s_kv = s_base;                                      // [stage][K, V]
  uint8_t* s_qd = s_kv + 2 * kStages * Sh::kTileBytes;         // [stage][Q, dO]
  uint8_t* s_ds = s_qd + 2 * kStages * Sh::kTileBytes;         // dS: key rows, a panel for each half of the queries
  float* s_col = reinterpret_cast<float*>(s_ds + 2 * kPanel);  // [-lse log2(e), -D][128 queries]
  using Item = ShortItem<!kBf16>;
  Item* s_item = reinterpret_cast<Item*>(s_col + 2 * kTile);
  uint64_t* s_bar = reinterpret_cast<uint64_t*>((reinterpret_cast<uintptr_t>(s_item + kItemRing) + 7) & ~(uintptr_t)7);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_bar + 32);
  volatile WaitState* s_wait = reinterpret_cast<volatile WaitState*>(s_tmem + 1);
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t kv_full = bars, kv_empty = bars + 16, qd_full = bars + 32, qd_empty = bars + 48, item_full = bars + 64,
                 item_empty = bars + 80, col_full = bars + 96, stored = bars + 104,
                 scores_full = bars + 112, ready = bars + 120, done = bars + 128, drain = bars + 136;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kv_full + 8 * i, 1);
      mbar_init(kv_empty + 8 * i, 1);
      mbar_init(qd_full + 8 * i, 1);
      mbar_init(qd_empty + 8 * i, 1);
      mbar_init(item_full + 8 * i, 1);
      mbar_init(item_empty + 8 * i, kSoftmaxThreads + 1);
    }
    mbar_init(col_full, kSoftmaxThreads);
    mbar_init(stored, kSoftmaxThreads);
    mbar_init(scores_full, 1);
    mbar_init(ready, kSoftmaxThreads);
    mbar_init(done, 1);
    mbar_init(drain, 1);
    s_wait->gave_up = 0;
    s_wait->polls = a.test.polls;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
    tma_prefetch_map(&map_do);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(s_tmem), Sh::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*s_tmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kLoadWarp) {
    // ------------------------------------------------ items and loads
    ItemClaims claims(&a.hdr->next_item[kShortEvents], a.items, a.kv_heads, a.hdr->n_items[kShortEvents]);
    int n = 0, u = 0;  // items and units with tiles so far
    bool ok = true;
    for (int i = 0; ok; ++i) {
      // The issuing warp looks one item ahead, so the ring holds none without
      // a pair: this warp clears their gradient rows itself.
      TileItem e;
      int h;
      bool more;
      while ((more = claims.take(&e, &h)) && (e.nq == 0 || e.nk == 0)) {
        clear_strided(static_cast<T*>(a.dq) + ((int64_t)e.q0 * a.heads + h * a.group) * a.D, e.nq,
                      (int64_t)a.heads * a.D, a.group * a.D);
        const int64_t at = ((int64_t)e.k0 * a.kv_heads + h) * a.D, stride = (int64_t)a.kv_heads * a.D;
        clear_strided(static_cast<T*>(a.dk) + at, e.nk, stride, a.D);
        clear_strided(static_cast<T*>(a.dv) + at, e.nk, stride, a.D);
      }
      const int slot = i % kItemRing;
      if (i >= kItemRing && !mbar_wait_warp(item_empty + 8 * slot, ((i / kItemRing) - 1) & 1, s_wait)) break;
      Item w;
      w.h = h;
      w.q_row = e.q0;
      w.nq = more ? e.nq : -1;
      w.k_row = e.k0;
      w.nk = e.nk;
      if constexpr (!kBf16) w.set(more ? range_scale(a.range[e.q0], a.range[a.n_q + e.q0]) : 1.f);
      if (lane == 0) s_item[slot] = w;
      __syncwarp();
      mbar_arrive_one(item_full + 8 * slot);
      if (!more) break;
      const int ks = n % kStages;
      if (n >= kStages && !mbar_wait_warp(kv_empty + 8 * ks, ((n / kStages) - 1) & 1, s_wait)) break;
      ++n;
      const auto load = [&](uint8_t* to, const CUtensorMap* m1, const CUtensorMap* m2, uint32_t bar, int rows, int row, int hd) {
        const int boxes = (rows + 63) / 64;
        mbar_expect(bar, 2 * boxes * 8192 * Sh::kPanels);
#pragma unroll 1
        for (int b = 0; b < boxes; ++b)
#pragma unroll
          for (int p = 0; p < Sh::kPanels; ++p) {
            const uint32_t at = smem_u32(to) + p * kPanel + b * 8192;
            tma_load(at, m1, bar, p * 64, hd, row + b * 64);
            tma_load(at + Sh::kTileBytes, m2, bar, p * 64, hd, row + b * 64);
          }
      };
      load(s_kv + 2 * ks * Sh::kTileBytes, &map_k, &map_v, kv_full + 8 * ks, e.nk, e.k0, h);
#pragma unroll 1
      for (int m = 0; m < a.group; ++m, ++u) {
        const int st = u % kStages;
        if (u >= kStages && !(ok = mbar_wait_warp(qd_empty + 8 * st, ((u / kStages) - 1) & 1, s_wait))) break;
        if ((a.test.skip & FPS_SKIP_SHORT) && blockIdx.x == 0 && u == 0) continue;
        load(s_qd + 2 * st * Sh::kTileBytes, &map_q, &map_do, qd_full + 8 * st, e.nq, e.q0, h * a.group + m);
      }
    }
    // after a wait that gave up: the copies still in flight land first
    if (__any_sync(kFull, s_wait->gave_up)) {
      for (int b = 0; b < kStages; ++b) {
        const int lk = n - 1 - b, lu = u - 1 - b;
        if (lk >= 0) mbar_land_warp(kv_full + 8 * (lk % kStages), (lk / kStages) & 1, s_wait);
        if (lu >= 0) mbar_land_warp(qd_full + 8 * (lu % kStages), (lu / kStages) & 1, s_wait);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ products
    const int cols = (a.D + 15) / 16 * 16;
    const uint32_t ts_desc = mma_desc(kBf16, false, true, cols);  // dV: A in TMEM; dK: dS along its rows
    const uint32_t dq_desc = mma_desc(kBf16, true, true, cols);   // dQ: dS across its rows
    const uint32_t dv_low = mma_desc(kBf16, false, true, min(cols, 32)), dv_high = mma_desc(kBf16, false, true, cols - 32);
    const uint32_t ds = smem_desc(smem_u32(s_ds), kPanel);
    int n = 0, u = 0;  // items and units so far
    bool ok = true;
    for (int i = 0; ok; ++i, ++n) {
      const int slot = i % kItemRing;
      if (!(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) break;
      const int nq = uniform(s_item[slot].nq), nk = uniform(s_item[slot].nk);
      mbar_arrive_one(item_empty + 8 * slot);
      if (nq < 0) break;
      const int ks = n % kStages;
      const uint32_t kv = smem_desc(smem_u32(s_kv) + 2 * ks * Sh::kTileBytes, kPanel);
      if (!(ok = mbar_wait_warp(kv_full + 8 * ks, (n / kStages) & 1, s_wait))) break;
      const uint32_t s_desc = mma_desc(kBf16, false, false, (nq + 15) / 16 * 16);
#pragma unroll 1
      for (int m = 0; m < a.group; ++m, ++u) {
        const int st = u % kStages;
        const uint32_t qd = smem_desc(smem_u32(s_qd) + 2 * st * Sh::kTileBytes, kPanel);
        if (!(ok = mbar_wait_warp(qd_full + 8 * st, (u / kStages) & 1, s_wait))) break;
        // the last unit's gradients lie where these scores go
        if (u > 0 && !(ok = mbar_wait_warp(stored, (u - 1) & 1, s_wait))) break;
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < 2; ++x)  // S, then dP: whole panels, as values past D are zeros
#pragma unroll
          for (int p = 0; p < Sh::kPanels; ++p)
            mma_ss<2, 2>(tmem + (x ? kColDP : kColS), kv + ((x * Sh::kTileBytes + p * kPanel) >> 4),
                         qd + ((x * Sh::kTileBytes + p * kPanel) >> 4), s_desc, p > 0);
        mma_commit(scores_full);
        if (!(ok = mbar_wait_warp(ready, u & 1, s_wait))) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half * 64 < nq; ++half) {  // 64 queries at a time
          const bool more = m > 0 || half > 0;
          const uint32_t q_rows = qd + half * kRun, do_rows = q_rows + (Sh::kTileBytes >> 4);
          const uint32_t p16 = tmem + kColS + half * 64;  // P lies over the first half of its scores
          if constexpr (kTwo) {  // dV += P^T dO
            mma_ts(tmem + kColS + 32, p16, do_rows, dv_low, more);
            if (cols > 32) mma_ts(tmem + kColS + 96, p16, do_rows + 4, dv_high, more);  // 32 values, 64 bytes on
          } else {
            mma_ts(tmem + Sh::kColDV, p16, do_rows, ts_desc, more);
          }
          mma_ss<2, 128>(tmem + Sh::kColDK, ds + half * (kPanel >> 4), q_rows, ts_desc, more);  // dK += dS^T Q
        }
#pragma unroll 1
        for (int half = 0; half * 64 < nk; ++half)  // dQ = dS K, 64 keys at a time
          mma_ss<128, 128>(tmem + Sh::kColDQ, ds + half * kRun, kv + half * kRun, dq_desc, half > 0);
        mma_commit(qd_empty + 8 * st);
        if (m == a.group - 1) mma_commit(kv_empty + 8 * ks);
        mma_commit(done);
      }
    }
    if (__any_sync(kFull, s_wait->gave_up)) {  // products in flight end before TMEM is freed
      mma_commit(drain);
      mbar_land_warp(drain, 0, s_wait);
    }
  } else {
    // ------------------------------------------------ softmax and its gradient
    const int half = warp >> 2, quarter = warp & 3;
    const int row = threadIdx.x & 127, h0 = half * kHalf;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    uint8_t* ds_row = s_ds + half * kPanel + row * 128;
    constexpr float kBackP = Item::kBackP;
    int n = 0, u = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int slot = i % kItemRing;
      if (!(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) break;
      const Item w = s_item[slot];
      if (w.nq < 0) break;
      mbar_arrive(item_empty + 8 * slot);
      T* dq = static_cast<T*>(a.dq) + (((int64_t)w.q_row + row) * a.heads + w.h * a.group) * a.D;
      const int64_t key_at = (((int64_t)w.k_row + row) * a.kv_heads + w.h) * a.D;
      const int shift = w.nk - w.nq, ks = n % kStages;
      const int q = warp * 16 + (lane >> 1);  // the query whose D this thread and the next form
      // the second of a pair of threads has no need of lse: where -D is there, it reads that
      const bool some_few = may_see_few(a.mask, w.nq, w.nk);
      const auto given = [&] { return some_few && (lane & 1) && few_keys(a.mask, q + shift, w.nk); };
      const ColumnSpan span = column_span(a.mask, row);
#pragma unroll 1
      for (int m = 0; m < a.group; ++m, ++u) {
        const int st = u % kStages, h = w.h * a.group + m;
        // D and lse of the unit's queries, two threads for each; O is on its
        // way while dO's tile is waited for
        uint4 o[DP / 16];
        float lse = 0.f, delta = 0.f;
        const int d0 = (lane & 1) * (DP / 16);
        if (q < w.nq) {
          const T* from = static_cast<const T*>(a.out) + (((int64_t)w.q_row + q) * a.heads + h) * a.D;
#pragma unroll
          for (int c = 0; c < DP / 16; ++c)
            o[c] = (d0 + c) * 8 < a.D ? *reinterpret_cast<const uint4*>(from + (d0 + c) * 8) : make_uint4(0, 0, 0, 0);
          lse = (given() ? a.rows + (int64_t)a.heads * a.n_q : a.lse)[(int64_t)h * a.n_q + w.q_row + q];
        }
        if (!(ok = mbar_wait_warp(qd_full + 8 * st, (u / kStages) & 1, s_wait))) break;
        uint8_t* tile = s_qd + 2 * st * Sh::kTileBytes;
        if (w.nq & 63) {
          clear_rows<Sh::kPanels>(tile, w.nq, w.nq, threadIdx.x, kSoftmaxThreads);
          clear_rows<Sh::kPanels>(tile + Sh::kTileBytes, w.nq, w.nq, threadIdx.x, kSoftmaxThreads);
        }
        if (m == 0 && (w.nk & 63)) {
          if (!(ok = mbar_wait_warp(kv_full + 8 * ks, (n / kStages) & 1, s_wait))) break;
          clear_rows<Sh::kPanels>(s_kv + 2 * ks * Sh::kTileBytes, w.nk, w.nk, threadIdx.x, kSoftmaxThreads);
        }
        if (q < w.nq) {
          const uint8_t* d = tile + Sh::kTileBytes + q * 128;
#pragma unroll
          for (int c = 0; c < DP / 16; ++c) {
            const int at = d0 + c;
            const uint4 vd = *reinterpret_cast<const uint4*>(d + (at >> 3) * kPanel + (((at & 7) ^ (q & 7)) << 4));
            const uint32_t* po = reinterpret_cast<const uint32_t*>(&o[c]);
            const uint32_t* pd = reinterpret_cast<const uint32_t*>(&vd);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = unpack16<T>(po[k]), y = unpack16<T>(pd[k]);
              delta = fmaf(x.x, y.x, fmaf(x.y, y.y, delta));
            }
          }
        }
        delta += __shfl_xor_sync(kFull, delta, 1);
        if constexpr (kBf16)
          s_col[(lane & 1) * kTile + q] = given() ? lse : lane & 1 ? -delta : -lse * kLog2e;
        else
          s_col[(lane & 1) * kTile + q] = lane & 1 ? (given() ? lse : -delta) * w.c : kWeightShift - lse * kLog2e;
        mbar_arrive(col_full);
        if (!(ok = mbar_wait_warp(scores_full, u & 1, s_wait))) break;
        if (!(ok = mbar_wait_warp(col_full, u & 1, s_wait))) break;
        tc_fence_after();
        // 32 queries at a time, to the end of this thread's 64 if there are any:
        // the products take P and dS of all of them
#pragma unroll 1
        for (int at = h0; at < h0 + kHalf && h0 < w.nq; at += 32) {
          uint32_t p16[16], d16[16];
          // which pairs of the warp's key rows and these queries see one another
          const int key = quarter * 32, pa = at + shift;
          if (at < w.nq && key < w.nk && some_seen(a.mask, pa, pa + 31, key)) {
            float x[32], y[32];
            tmem_ld32(lanes + kColS + at, reinterpret_cast<uint32_t*>(x));
            tmem_ld32(lanes + kColDP + at, reinterpret_cast<uint32_t*>(y));
            tmem_wait_ld32(reinterpret_cast<uint32_t*>(x));
            tmem_wait_ld32(reinterpret_cast<uint32_t*>(y));
            const float* col = s_col + at;
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 le = *reinterpret_cast<const float4*>(col + k);
              const float4 de = *reinterpret_cast<const float4*>(col + kTile + k);
              const float2 e0 = fma2(make_float2(x[k], x[k + 1]), scale2, make_float2(le.x, le.y));
              const float2 e1 = fma2(make_float2(x[k + 2], x[k + 3]), scale2, make_float2(le.z, le.w));
              x[k] = exp2_approx(e0.x);
              x[k + 1] = exp2_approx(e0.y);
              x[k + 2] = exp2_approx(e1.x);
              x[k + 3] = exp2_approx(e1.y);
              const uint64_t p0 = pack2(y[k], y[k + 1]), p1 = pack2(y[k + 2], y[k + 3]);
              const uint64_t d0 = pack2(de.x, de.y), d1 = pack2(de.z, de.w), c2 = pack2(w.c, w.c);
              const uint64_t y0 = mul2(kBf16 ? add2(p0, d0) : fma2(p0, c2, d0), pack2(x[k], x[k + 1]));
              const uint64_t y1 = mul2(kBf16 ? add2(p1, d1) : fma2(p1, c2, d1), pack2(x[k + 2], x[k + 3]));
              y[k] = lo2(y0);
              y[k + 1] = hi2(y0);
              y[k + 2] = lo2(y1);
              y[k + 3] = hi2(y1);
            }
            if (at + 32 > w.nq || key + 32 > w.nk || !all_seen(a.mask, pa, pa + 31, key)) {
              const uint32_t see = row < w.nk ? bits(0, w.nq - at) & bits(span.lo - pa, span.hi + 1 - pa) : 0u;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see >> k & 1)) x[k] = y[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              p16[k] = pack16<T>(x[2 * k], x[2 * k + 1]);
              d16[k] = pack16<T>(y[2 * k], y[2 * k + 1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) p16[k] = d16[k] = 0;
          }
          tmem_st16(lanes + kColS + h0 + (at - h0) / 2, p16);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(ds_row + ((((at - h0) / 8 + k) ^ (row & 7)) << 4)) =
                make_uint4(d16[4 * k], d16[4 * k + 1], d16[4 * k + 2], d16[4 * k + 3]);
        }
        tmem_wait_st();
        fence_async_smem();  // dS, and the cleared rows
        tc_fence_before();
        mbar_arrive(ready);
        // stores: dQ of this head, half of the columns each; after the last
        // head dK and dV
        if (!(ok = mbar_wait_warp(done, u & 1, s_wait))) break;
        tc_fence_after();
        const float back = a.scale * w.back;  // of dQ and dK
        store_row<T, DP / 2>(lanes + Sh::kColDQ + half * (DP / 2), row < w.nq, back, dq + m * a.D + half * (DP / 2),
                             a.D - half * (DP / 2), a.sectors);
        if (kTwo) {  // half of dV's columns are in each half of the scores
          store_row<T, 32>(lanes + Sh::kColDK + half * 32, row < w.nk, back, static_cast<T*>(a.dk) + key_at + half * 32,
                           a.D - half * 32, a.sectors);
          store_row<T, 32>(lanes + kColS + 32 + half * 64, row < w.nk, kBackP, static_cast<T*>(a.dv) + key_at + half * 32,
                           a.D - half * 32, a.sectors);
        } else if (m == a.group - 1) {
          store_row<T, DP>(lanes + (half == 0 ? Sh::kColDK : Sh::kColDV), row < w.nk, half == 0 ? back : kBackP,
                           static_cast<T*>(half == 0 ? a.dk : a.dv) + key_at, a.D, a.sectors);
        }
        tc_fence_before();
        mbar_arrive(stored);
      }
      ++n;
    }
  }
  if (rows_known(a.hdr)) {
    zero_rows(a.dq, a.B > 0 ? a.q_offsets[a.B] : 0, a.n_q, (int64_t)a.heads * a.D);
    zero_rows(a.dk, a.B > 0 ? a.kv_offsets[a.B] : 0, a.n_kv, (int64_t)a.kv_heads * a.D);
    zero_rows(a.dv, a.B > 0 ? a.kv_offsets[a.B] : 0, a.n_kv, (int64_t)a.kv_heads * a.D);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, Sh::kColumns);
  }
  if (threadIdx.x == 0 && s_wait->gave_up) record_error(a.hdr, kDevWaitTimeout);
}

template <typename T, int DP, bool kTwo>
cudaError_t run(const ShortArgs& a, const BwdMaps& m, cudaStream_t s) {
  const auto kernel = k_attn_backward_short<T, DP, kTwo>;
  constexpr int smem = (int)ShortShape<DP, kTwo>::kSmem;
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.B * a.kv_heads, slots = (int64_t)device_info().sm_count * (kTwo ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < slots ? items : slots));
  cfg.blockDim = dim3(kShortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a, m.q, m.k, m.v, m.d);
}

template <typename T>
cudaError_t run_type(const ShortArgs& a, const BwdMaps& m, cudaStream_t s) {
  if (a.D > 64) return run<T, 128, false>(a, m, s);
  return a.group == 1 ? run<T, 64, true>(a, m, s) : run<T, 64, false>(a, m, s);
}

}  // namespace

cudaError_t launch_attention_backward_short(const AttnCall& c, const BwdMaps& maps, const float* rows, const float* range,
                                            const TileItem* items, WsHeader* hdr, cudaStream_t s) {
  ShortArgs a;
  a.n_q = c.n_q;
  a.n_kv = c.n_kv;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.group = c.group;
  a.D = c.D;
  a.mask = c.mask;
  a.scale = c.scale;
  a.scale_log2 = c.scale * kLog2e;
  a.out = c.out;
  a.lse = c.lse;
  a.rows = rows;
  a.range = range;
  a.dq = c.dq;
  a.dk = c.dk;
  a.dv = c.dv;
  a.q_offsets = c.q_offsets;
  a.kv_offsets = c.kv_offsets;
  a.B = c.B;
  a.test = c.test;
  a.sectors = maps.sectors;
  a.items = items;
  a.hdr = hdr;
  return c.dtype == FPS_DTYPE_BF16 ? run_type<__nv_bfloat16>(a, maps, s) : run_type<__half>(a, maps, s);
}

}  // namespace fpstok
