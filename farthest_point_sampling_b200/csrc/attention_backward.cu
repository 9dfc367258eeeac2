// Attention of packed events, backward, on the tensor cores.
//
// With S, P and lse of the forward and D_i = sum_d dO_id O_id,
//   dV = P^T dO,   dP = dO V^T,   dS = P (dP - D),   dQ = scale dS K,   dK = scale dS^T Q,
// the K and V gradients summed over the query heads that share them.
//
// Two kernels, one template.  A work item keeps a 128-row tile of one pair of
// tensors and streams tiles of the other past it:
//   queries: keeps Q, dO of one query tile and head, streams K, V:
//            scores S = Q K^T and dP = dO V^T, then dQ += dS K;
//   keys:    keeps K, V of one key tile and key head, streams Q, dO of every
//            query tile that sees it, for every head of the group:
//            S^T = K Q^T and dP^T = V dO^T, then dV += P^T dO, dK += dS^T Q.
// P is formed again from the scores and lse.  Each gradient tile is summed by
// one block in a fixed order, so the result does not depend on scheduling;
// the price is that the scores are formed twice.
//
// A key tile that every query of a long event sees - the first keys under
// `sinks`, or all without a window - is as much work as its event is long, and
// one block would end last with it.  Such tiles are cut into pieces of their
// (head, query tile) range; each piece leaves float32 sums, and a second kernel
// adds a tile's pieces in order.  64 track events of up to 20000 tokens (causal
// window of 511, 4 sinks, 8 query and 2 key heads of 128): a sixth less time than
// with whole tiles.
//
// Roles as in the forward kernel: a loading warp, an issuing warp, and softmax
// warps with a thread for each kept row and 64 streamed rows.  P and dS go
// back to TMEM as 16-bit operand A, each over the scores its thread read.  The
// products of a tile are spread under the softmax of it and the next: S of
// tile m + 1 runs while dS of tile m is formed, then dK of m and dP of m + 1
// run while the weights of m + 1 are.
//
// Streamed tiles are 128 rows for 128-wide heads, whose accumulators take half
// of an SM's TMEM: one block with eight softmax warps has it all.  For 64-wide
// heads they are 64 rows, and two blocks share an SM, each with four softmax
// warps and 256 columns: where events are a few tiles long one block's loads
// and stores then run under the other's products (2048 events of up to 256
// tokens, 8 heads of 64; tiles and blocks as for 128 took a fifth longer).
// Where two sets of accumulators fit, a block goes on with the next item while
// it stores one.
//
// What bounds it: the softmax side.  4 causal events of 4000 to 9000 tokens, 16
// query and 4 key heads of 128: 2.46 ms, 662 TFLOP/s of five products (seven are
// done), where the five would take 0.98 ms; the two kernels form each weight
// twice and each holds a thread's 64 scores in registers between TMEM reads and
// writes.  Short items add the latency of filling the pipeline: 2048 events of up
// to 256 tokens, 8 heads of 64: 1.78 ms with the kernel of the short ones, 2.0
// TB/s.
//
// Rounding: P and dS are rounded to the input type for their products, in
// float16 scaled into its range (attention_backward_range.cu).  D
// comes from the rounded output, as the forward left it, but for queries that
// see few keys, where that would show (attention_backward_rows.cu).
#include <type_traits>

#include "attention_few.h"
#include "attention_plan.h"
#include "attention_short.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace fpstok {

namespace {

constexpr int kRows = 64;                     // streamed rows that a thread takes
constexpr int kPanel = kTile * 128;           // bytes of a kept tile's 64-value panel
constexpr int kItemRing = 2;

struct BwdArgs {
  int64_t n_q, n_kv;
  int heads, kv_heads, group, D;
  AttnMask mask;
  float scale, scale_log2;
  const void* out;
  const float* lse;
  // [2][heads, n_q]: -lse log2(e) and -D (float16: the one 14 more, the other
  // times the event's c), written by the queries kernel for the keys kernel; of
  // queries that see few keys -D is there before
  float* rows;
  const float* range;  // float16: see attention_backward_range.cu
  float* partial;  // [slot][key head][128][2 DP]: dK and dV of the pieces of a key tile
  void* d1;      // dQ, or dK
  void* d2;      // dV
  WaitTest test;
  bool sectors;  // every gradient row starts on a 32-byte sector, and ends on one
  const TileItem* items;
  WsHeader* hdr;
};

// One work item as the loading warp hands it to the others.
template <int kStream, bool kScaled>
struct BwdItem : ItemScale<kScaled> {
  int count;            // streamed tiles of one head; -1 ends the work
  int f0, f1;           // which of those of all heads in turn this item takes
  int hd, j;            // the first one's head in the group, and its place among the head's
  int slot;             // where its sums go: -1 for the gradients
  int h;                // head (queries kernel) or key head
  int kept_row, rows;   // first kept row, how many
  int at;               // the first kept row in its event
  int stream_row, stream_rows;  // the event's first streamed row, and how many it has
  int shift;            // nk - nq: position of query 0
  KeyTiles<kStream> tiles;
};
template <bool kKeys, bool kScaled, int kStream>
__device__ __forceinline__ BwdItem<kStream, kScaled> bwd_item(const BwdArgs& a, int h, const TileItem& e) {
  BwdItem<kStream, kScaled> w;
  w.h = h;
  w.at = e.t * kTile;
  w.kept_row = (kKeys ? e.k0 : e.q0) + w.at;
  w.rows = min(kTile, (kKeys ? e.nk : e.nq) - w.at);
  w.stream_row = kKeys ? e.q0 : e.k0;
  w.stream_rows = kKeys ? e.nq : e.nk;
  w.shift = e.nk - e.nq;
  if constexpr (kKeys) {
    int lo, hi;
    queries_of(a.mask, w.at, w.rows, w.shift, e.nq, &lo, &hi);
    w.tiles.before = w.tiles.s = 0;
    w.tiles.first = lo & ~15;
    w.tiles.end = hi;
    w.tiles.count = hi > lo ? (hi - w.tiles.first + kStream - 1) / kStream : 0;
  } else {
    w.tiles = key_tiles<kStream>(a.mask, w.at + w.shift, w.at + w.rows - 1 + w.shift, e.nk);
  }
  w.count = w.tiles.count;
  w.f0 = 0;
  w.f1 = w.count * (kKeys ? a.group : 1);
  w.slot = -1;
  w.hd = w.j = 0;
  if constexpr (kScaled)  // no pair, maybe no first query, and no use of it
    w.set(w.count > 0 ? range_scale(a.range[e.q0], a.range[a.n_q + e.q0]) : 1.f);
  if (kKeys && e.pad[2] != -1) {  // a piece
    w.f0 = e.pad[0];
    w.f1 = e.pad[1];
    w.slot = e.pad[2];
    if (w.f1 > w.f0) {
      w.hd = w.f0 / w.count;
      w.j = w.f0 - w.hd * w.count;
    }
  }
  return w;
}

template <int DP, bool kKeys>
struct BwdShape {
  static constexpr int kPanels = DP / 64;
  static constexpr int kBlocks = DP == 64 ? 2 : 1;
  static constexpr int kStream = DP == 64 ? 64 : 128;  // rows of a streamed tile
  static constexpr int kParts = kStream / kRows;       // threads of a kept row
  static constexpr int kSoftmaxThreads = kTile * kParts;
  static constexpr int kThreads = kSoftmaxThreads + 64;
  static constexpr uint32_t kKeptBytes = kPanels * kPanel;           // one kept tensor's tile
  static constexpr uint32_t kStreamPanel = kStream * 128;
  static constexpr uint32_t kStreamBytes = kPanels * kStreamPanel;   // one streamed tensor's tile
  // 96 KB for each of two blocks, or 192 KB for one
  static constexpr int kKept = DP == 64 ? 2 : 1;
  static constexpr int kRing = 2;
  static constexpr uint32_t kColS = 0, kColDP = kStream, kColAcc = 2 * kStream;
  static constexpr uint32_t kAccColumns = (kKeys ? 2 : 1) * DP;
  static constexpr uint32_t kColumns = 512 / kBlocks;
  static constexpr int kAcc = kColAcc + 2 * kAccColumns <= kColumns ? 2 : 1;
  static constexpr size_t kColFloats = kRing * 2 * kStream > 2 * kTile ? kRing * 2 * kStream : 2 * kTile;
  static constexpr size_t kSmem = 1024 + 2 * (kKept * kKeptBytes + kRing * kStreamBytes) + kColFloats * sizeof(float) +
                                  kItemRing * sizeof(BwdItem<kStream, true>) + 512;
};

// 4 bytes from global to shared memory, asynchronously; zero where not real.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool real) {
  const int n = real ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// One arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <typename T, int DP, bool kKeys>
__global__ void __launch_bounds__(BwdShape<DP, kKeys>::kThreads, BwdShape<DP, kKeys>::kBlocks)
    k_attn_backward(const BwdArgs a, const __grid_constant__ CUtensorMap map_k1, const __grid_constant__ CUtensorMap map_k2,
                    const __grid_constant__ CUtensorMap map_s1, const __grid_constant__ CUtensorMap map_s2) {
  using Sh = BwdShape<DP, kKeys>;
  using Item = BwdItem<Sh::kStream, !std::is_same<T, __nv_bfloat16>::value>;
  constexpr int kStream = Sh::kStream, kSoftmaxThreads = Sh::kSoftmaxThreads;
  constexpr uint32_t kColS = Sh::kColS, kColDP = Sh::kColDP, kColAcc = Sh::kColAcc;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kLoadWarp = kSoftmaxThreads / 32, kMmaWarp = kLoadWarp + 1;
  extern __shared__ uint8_t s_raw[];
  uint8_t* s_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  // kept tiles (tensor 1 and 2 of a stage side by side), then the streamed
  // ring, then the ring's -lse log2(e) and -D of its queries (keys kernel), or
  // those of the kept rows (queries kernel)
  uint8_t* s_kept = s_base;
  uint8_t* s_ring = s_kept + 2 * Sh::kKept * Sh::kKeptBytes;
  float* s_col = reinterpret_cast<float*>(s_ring + 2 * Sh::kRing * Sh::kStreamBytes);
  Item* s_item = reinterpret_cast<Item*>(s_col + Sh::kColFloats);
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_item + kItemRing);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_bar + 32);
  volatile WaitState* s_wait = reinterpret_cast<volatile WaitState*>(s_tmem + 1);
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t kept_full = bars, kept_empty = bars + 16, acc_full = bars + 32, acc_empty = bars + 48,
                 item_full = bars + 64, item_empty = bars + 80, s_full = bars + 96, dp_full = bars + 104,
                 p_ready = bars + 112, ds_ready = bars + 120, drain = bars + 128, ring_full = bars + 136,
                 ring_empty = bars + 168, row_ready = bars + 208, dv_done = bars + 216;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kept_full + 8 * i, 1);
      // in the queries kernel the softmax threads read the kept dO themselves
      mbar_init(kept_empty + 8 * i, kKeys ? 1 : 1 + kSoftmaxThreads);
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, kSoftmaxThreads);
      mbar_init(item_full + 8 * i, 1);
      mbar_init(item_empty + 8 * i, kSoftmaxThreads + 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, kSoftmaxThreads);
    mbar_init(ds_ready, kSoftmaxThreads);
    mbar_init(drain, 1);
    mbar_init(row_ready, kSoftmaxThreads);
    mbar_init(dv_done, 1);
    for (int i = 0; i < Sh::kRing; ++i) {
      mbar_init(ring_full + 8 * i, kKeys ? 33 : 1);  // the tiles, and in the keys kernel each lane's -lse and -D
      mbar_init(ring_empty + 8 * i, 1);
    }
    s_wait->gave_up = 0;
    s_wait->polls = a.test.polls;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_k1);
    tma_prefetch_map(&map_k2);
    tma_prefetch_map(&map_s1);
    tma_prefetch_map(&map_s2);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(s_tmem), Sh::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*s_tmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kLoadWarp) {
    // ------------------------------------------------ items and loads
    constexpr int kList = kKeys ? kKeyTiles : kQueryTiles;
    ItemClaims claims(&a.hdr->next_item[kList], a.items, kKeys ? a.kv_heads : a.heads, a.hdr->n_items[kList]);
    int i = 0, n = 0, nk = 0;  // items handed out, streamed and kept tiles loaded so far
    bool ok = true;
    for (; ok; ++i) {
      // The issuing warp looks one item ahead, so the ring holds none without
      // tiles: this warp clears their gradient rows itself.
      TileItem entry;
      Item w;
      int h;
      bool more;
      while ((more = claims.take(&entry, &h))) {
        w = bwd_item<kKeys, !kBf16, kStream>(a, h, entry);
        if (w.slot == -2) continue;
        if (w.f1 > w.f0) break;
        const int heads = kKeys ? a.kv_heads : a.heads;
        const int64_t at = ((int64_t)w.kept_row * heads + h) * a.D, stride = (int64_t)heads * a.D;
        clear_strided(static_cast<T*>(a.d1) + at, w.rows, stride, a.D);
        if (kKeys) clear_strided(static_cast<T*>(a.d2) + at, w.rows, stride, a.D);
      }
      const int slot = i % kItemRing;
      if (i >= kItemRing && !mbar_wait_warp(item_empty + 8 * slot, ((i / kItemRing) - 1) & 1, s_wait)) break;
      if (!more) {
        if (lane == 0) s_item[slot].count = -1;
        __syncwarp();
        mbar_arrive_one(item_full + 8 * slot);
        break;
      }
      if (lane == 0) s_item[slot] = w;
      __syncwarp();
      mbar_arrive_one(item_full + 8 * slot);
      const int ks = nk % Sh::kKept;
      if (nk >= Sh::kKept && !mbar_wait_warp(kept_empty + 8 * ks, ((nk / Sh::kKept) - 1) & 1, s_wait)) break;
      const int boxes = (w.rows + 63) / 64;
      const bool skip = (a.test.skip & (kKeys ? FPS_SKIP_KEYS : FPS_SKIP_QUERIES)) && blockIdx.x == 0 && nk == 0;
      if (!skip) mbar_expect(kept_full + 8 * ks, 2 * boxes * 8192 * Sh::kPanels);
#pragma unroll 1
      for (int b = 0; b < (skip ? 0 : boxes); ++b)
#pragma unroll
        for (int p = 0; p < Sh::kPanels; ++p) {
          const uint32_t to = smem_u32(s_kept) + 2 * ks * Sh::kKeptBytes + p * kPanel + b * 8192;
          tma_load(to, &map_k1, kept_full + 8 * ks, p * 64, w.h, w.kept_row + b * 64);
          tma_load(to + Sh::kKeptBytes, &map_k2, kept_full + 8 * ks, p * 64, w.h, w.kept_row + b * 64);
        }
      ++nk;
      const int head0 = kKeys ? w.h * a.group : w.h / a.group;
      int hd = w.hd, j = w.j;
#pragma unroll 1
      for (int f = w.f0; f < w.f1; ++f, ++n) {
        const int st = n % Sh::kRing;
        if (n >= Sh::kRing && !(ok = mbar_wait_warp(ring_empty + 8 * st, ((n / Sh::kRing) - 1) & 1, s_wait))) break;
        const int row = w.stream_row + w.tiles.start(j), extent = w.tiles.extent(j);
        const int sboxes = (extent + 63) / 64;
        mbar_expect(ring_full + 8 * st, 2 * sboxes * 8192 * Sh::kPanels);
#pragma unroll 1
        for (int b = 0; b < sboxes; ++b)
#pragma unroll
          for (int p = 0; p < Sh::kPanels; ++p) {
            const uint32_t to = smem_u32(s_ring) + 2 * st * Sh::kStreamBytes + p * Sh::kStreamPanel + b * 8192;
            tma_load(to, &map_s1, ring_full + 8 * st, p * 64, head0 + hd, row + b * 64);
            tma_load(to + Sh::kStreamBytes, &map_s2, ring_full + 8 * st, p * 64, head0 + hd, row + b * 64);
          }
        if constexpr (kKeys) {
          const float* from = a.rows + (int64_t)(head0 + hd) * a.n_q + row;
          const uint32_t to = smem_u32(s_col + st * 2 * kStream);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int c = lane; c < kStream; c += 32)
              copy4(to + (x * kStream + c) * 4, from + (c < extent ? (int64_t)x * a.heads * a.n_q + c : 0), c < extent);
          copy_arrive(ring_full + 8 * st);
        }
        if (++j == w.count) {
          j = 0;
          ++hd;
        }
      }
    }
    // after a wait that gave up: the copies still in flight land first
    if (__any_sync(kFull, s_wait->gave_up)) {
      for (int b = 0; b < Sh::kRing; ++b) {
        const int lk = nk - 1 - b, ls = n - 1 - b;
        if (lk >= 0 && b < Sh::kKept) mbar_land_warp(kept_full + 8 * (lk % Sh::kKept), (lk / Sh::kKept) & 1, s_wait);
        if (ls >= 0) mbar_land_warp(ring_full + 8 * (ls % Sh::kRing), (ls / Sh::kRing) & 1, s_wait);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ products
    const uint32_t out_desc = mma_desc(kBf16, false, true, (a.D + 15) / 16 * 16);
    // The next tile in the order of the work, across items: its item's kept
    // stage and accumulators, and whether it is the item's first and last.
    struct Tile {
      int steps, kept, item;
      bool first, last;
    };
    int i = 0, f = 0, f0 = 0, f1 = 0, j = 0, count = 0, items = 0, fetched = 0;  // items and tiles read, place in the item
    KeyTiles<kStream> tiles = {};
    bool ok = true;
    const auto fetch = [&](Tile* t) {  // false when the work is done, or a wait gave up (ok)
      if (f == f1) {
        const int slot = i % kItemRing;
        if (!(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) return false;
        count = uniform(s_item[slot].count);
        f0 = f = uniform(s_item[slot].f0);
        f1 = uniform(s_item[slot].f1);
        j = uniform(s_item[slot].j);
        tiles.before = uniform(s_item[slot].tiles.before);
        tiles.first = uniform(s_item[slot].tiles.first);
        tiles.end = uniform(s_item[slot].tiles.end);
        tiles.s = uniform(s_item[slot].tiles.s);
        mbar_arrive_one(item_empty + 8 * slot);
        if (count < 0) return false;
        ++i;
        const int ks = items % Sh::kKept;
        if (!(ok = mbar_wait_warp(kept_full + 8 * ks, (items / Sh::kKept) & 1, s_wait))) return false;
        ++items;
      }
      const int st = fetched % Sh::kRing;
      if (!(ok = mbar_wait_warp(ring_full + 8 * st, (fetched / Sh::kRing) & 1, s_wait))) return false;
      ++fetched;
      t->steps = (tiles.extent(j) + 15) / 16;
      t->item = items - 1;
      t->kept = t->item % Sh::kKept;
      t->first = f == f0;
      t->last = ++f == f1;
      if (++j == count) j = 0;
      tc_fence_after();
      return true;
    };
    // S (x = 0) or dP (x = 1) of tile m: a kept and a streamed tensor; whole
    // panels, as values past D are zeros
    const auto scores = [&](const Tile& t, int m, int x) {
      const uint32_t kept = smem_desc(smem_u32(s_kept) + (2 * t.kept + x) * Sh::kKeptBytes, kPanel);
      const uint32_t from = smem_desc(smem_u32(s_ring) + (2 * (m % Sh::kRing) + x) * Sh::kStreamBytes, Sh::kStreamPanel);
      const uint32_t desc = mma_desc(kBf16, false, false, t.steps * 16);
#pragma unroll
      for (int p = 0; p < Sh::kPanels; ++p)
        mma_ss<2, 2>(tmem + (x ? kColDP : kColS), kept + p * (kPanel >> 4), from + p * (Sh::kStreamPanel >> 4), desc, p > 0);
      mma_commit(x ? dp_full : s_full);
    };
    // an accumulator += the 16-bit rows over S or dP, times a streamed tensor;
    // each 64 of the rows lie over the first half of their scores
    const auto gradient = [&](const Tile& t, int m, uint32_t from, uint32_t to, int x) {
      const uint32_t rows = smem_desc(smem_u32(s_ring) + (2 * (m % Sh::kRing) + x) * Sh::kStreamBytes, Sh::kStreamPanel);
      mma_ts(to, from, rows, out_desc, !t.first);
      if (Sh::kParts > 1 && t.steps > 4) mma_ts(to, from + kRows, rows + kRun, out_desc, true);
    };
    Tile cur, nxt;
    bool more = fetch(&cur);
    if (more) {
      scores(cur, 0, 0);
      scores(cur, 0, 1);
      if (cur.last) mma_commit(kept_empty + 8 * cur.kept);
    }
    for (int m = 0; more; ++m) {
      const uint32_t to = tmem + kColAcc + (cur.item % Sh::kAcc) * Sh::kAccColumns;
      if (cur.first && cur.item >= Sh::kAcc &&
          !mbar_wait_warp(acc_empty + 8 * (cur.item % Sh::kAcc), ((cur.item / Sh::kAcc) - 1) & 1, s_wait))
        break;
      if (!mbar_wait_warp(p_ready, m & 1, s_wait)) break;
      tc_fence_after();
      // Products of different shapes are not promised to run in order: scores
      // wait for the product that reads the 16-bit rows in their place.
      if constexpr (kKeys) {
        gradient(cur, m, tmem + kColS, to + DP, 1);  // dV += P^T dO
        mma_commit(dv_done);
      }
      more = fetch(&nxt);
      if (!ok) break;
      if (kKeys && !mbar_wait_warp(dv_done, m & 1, s_wait)) break;
      if (more) scores(nxt, m + 1, 0);
      if (!mbar_wait_warp(ds_ready, m & 1, s_wait)) break;
      tc_fence_after();
      gradient(cur, m, tmem + kColDP, to, 0);  // dK += dS^T Q, or dQ += dS K
      mma_commit(ring_empty + 8 * (m % Sh::kRing));
      if (cur.last) mma_commit(acc_full + 8 * (cur.item % Sh::kAcc));
      if (more) {
        if (!mbar_wait_warp(ring_empty + 8 * (m % Sh::kRing), (m / Sh::kRing) & 1, s_wait)) break;
        scores(nxt, m + 1, 1);
        if (nxt.last) mma_commit(kept_empty + 8 * nxt.kept);  // only the scores read the kept tiles
        cur = nxt;
      }
    }
    if (__any_sync(kFull, s_wait->gave_up)) {  // products in flight end before TMEM is freed
      mma_commit(drain);
      mbar_land_warp(drain, 0, s_wait);
    }
  } else {
    // ------------------------------------------------ softmax and its gradient
    const int part = warp >> 2, quarter = warp & 3;
    const int row = threadIdx.x & 127, h0 = part * kRows;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    int m = 0, nk = 0;
    bool ok = true;
    // Queries kernel: two threads read the row of O that belongs to a query of
    // the next item, before they store this one's gradients.
    constexpr int kOwn = 2 / Sh::kParts;  // queries of a pair of threads, 64 apart
    const int q0 = warp * 16 + (lane >> 1), d0 = (lane & 1) * (DP / 16);
    uint4 o[kOwn][DP / 16];
    float lse[kOwn] = {};
    bool given[kOwn] = {};
    const auto ahead = [&](int i) {
      if (!mbar_wait_warp(item_full + 8 * (i % kItemRing), (i / kItemRing) & 1, s_wait)) return false;
      const Item& w = s_item[i % kItemRing];
      if (w.count <= 0) return true;
#pragma unroll
      for (int r = 0; r < kOwn; ++r) {
        const int q = q0 + 64 * r;
        if (q >= w.rows) continue;
        // the second of the two has no need of lse: where -D is there, it reads that
        given[r] = (lane & 1) && few_keys(a.mask, w.at + q + w.shift, w.stream_rows);
        lse[r] = (given[r] ? a.rows + (int64_t)a.heads * a.n_q : a.lse)[(int64_t)w.h * a.n_q + w.kept_row + q];
        const T* from = static_cast<const T*>(a.out) + (((int64_t)w.kept_row + q) * a.heads + w.h) * a.D;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c)
          o[r][c] = (d0 + c) * 8 < a.D ? *reinterpret_cast<const uint4*>(from + (d0 + c) * 8) : make_uint4(0, 0, 0, 0);
      }
      return true;
    };
    if constexpr (!kKeys) ok = ahead(0);
    for (int i = 0; ok; ++i) {
      const int slot = i % kItemRing;
      if (kKeys && !(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) break;
      const Item& w = s_item[slot];  // read where it is needed: it stays until this thread lets go of the slot
      const int count = w.count;
      if (count < 0) break;
      float lse2 = 0.f, delta = 0.f;  // -lse log2(e) and -D of this thread's query, as in a.rows
      const uint64_t c2 = pack2(w.c, w.c);
      if constexpr (!kKeys) {
        // D: O as read ahead, dO from its tile; shared with the keys kernel
        // through memory and with the threads of each row through the block's
        const int ks = nk % Sh::kKept;
        if (!(ok = mbar_wait_warp(kept_full + 8 * ks, (nk / Sh::kKept) & 1, s_wait))) break;
#pragma unroll
        for (int r = 0; r < kOwn; ++r) {
          const int q = q0 + 64 * r;
          float sum = 0.f;
          if (q < w.rows) {
            const uint8_t* d = s_kept + (2 * ks + 1) * Sh::kKeptBytes + q * 128;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
              const int at = d0 + c;
              const uint4 vd = *reinterpret_cast<const uint4*>(d + (at >> 3) * kPanel + (((at & 7) ^ (q & 7)) << 4));
              const uint32_t* po = reinterpret_cast<const uint32_t*>(&o[r][c]);
              const uint32_t* pd = reinterpret_cast<const uint32_t*>(&vd);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 x = unpack16<T>(po[k]), y = unpack16<T>(pd[k]);
                sum = fmaf(x.x, y.x, fmaf(x.y, y.y, sum));
              }
            }
          }
          sum += __shfl_xor_sync(kFull, sum, 1);
          float mine;
          if constexpr (kBf16)
            mine = given[r] ? lse[r] : lane & 1 ? -sum : -lse[r] * kLog2e;
          else
            mine = lane & 1 ? (given[r] ? lse[r] : -sum) * w.c : kWeightShift - lse[r] * kLog2e;
          s_col[(lane & 1) * kTile + q] = mine;
          if (q < w.rows) a.rows[((int64_t)(lane & 1) * a.heads + w.h) * a.n_q + w.kept_row + q] = mine;
        }
        mbar_arrive(kept_empty + 8 * ks);
        mbar_arrive(row_ready);
        if (!(ok = mbar_wait_warp(row_ready, nk & 1, s_wait))) break;
        lse2 = s_col[row];
        delta = s_col[kTile + row];
      }
      const int f1 = w.f1;
#pragma unroll 1
      for (int f = w.f0, j = w.j; f < f1; ++f, ++m) {
        const int st = m % Sh::kRing;
        const int extent = w.tiles.extent(j), stream0 = w.tiles.start(j);
        j = j + 1 == count ? 0 : j + 1;
        const int left = w.stream_rows - stream0;
        const bool clear = rows_to_clear(extent, left);
        if (kKeys || clear) {
          // also where -lse and -D are read from
          if (!(ok = mbar_wait_warp(ring_full + 8 * st, (m / Sh::kRing) & 1, s_wait))) break;
        }
        if (clear) {
          uint8_t* tile = s_ring + 2 * st * Sh::kStreamBytes;
          clear_rows<Sh::kPanels, kStream>(tile, extent, left, threadIdx.x, kSoftmaxThreads);
          if (kKeys) clear_rows<Sh::kPanels, kStream>(tile + Sh::kStreamBytes, extent, left, threadIdx.x, kSoftmaxThreads);
          fence_async_smem();
        }
        // which pairs of the warp's kept rows and each 32 of this thread's
        // streamed rows see one another: some, all, and those of this thread's row
        bool act[2], whole[2];
        uint32_t see[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = h0 + 32 * c, r0 = w.at + quarter * 32, c0 = stream0 + at;
          const int pa = (kKeys ? c0 : r0) + w.shift, key = kKeys ? r0 : c0;
          act[c] = at < extent && some_seen(a.mask, pa, pa + 31, key);
          whole[c] = at + 32 <= extent && all_seen(a.mask, pa, pa + 31, key);
          if (act[c] && !whole[c]) {
            see[c] = bits(0, extent - at);
            if constexpr (kKeys) {
              const ColumnSpan span = column_span(a.mask, key + lane);
              see[c] &= bits(span.lo - pa, span.hi + 1 - pa);
            } else {
              see[c] &= seen_keys(a.mask, pa + lane, key);
            }
          }
        }
        const float* col = s_col + st * 2 * kStream + h0;
        if (!(ok = mbar_wait_warp(s_full, m & 1, s_wait))) break;
        tc_fence_after();
        float x[kRows];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32(lanes + kColS + h0 + 32 * c, reinterpret_cast<uint32_t*>(x + 32 * c));
        tmem_wait_ld32(reinterpret_cast<uint32_t*>(x));
        tmem_wait_ld32(reinterpret_cast<uint32_t*>(x + 32));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (act[c]) {
#pragma unroll
            for (int k = 32 * c; k < 32 * c + 32; k += 4) {
              float4 le = make_float4(lse2, lse2, lse2, lse2);
              if constexpr (kKeys) le = *reinterpret_cast<const float4*>(col + k);
              const float2 e0 = fma2(make_float2(x[k], x[k + 1]), scale2, make_float2(le.x, le.y));
              const float2 e1 = fma2(make_float2(x[k + 2], x[k + 3]), scale2, make_float2(le.z, le.w));
              x[k] = exp2_approx(e0.x);
              x[k + 1] = exp2_approx(e0.y);
              x[k + 2] = exp2_approx(e1.x);
              x[k + 3] = exp2_approx(e1.y);
            }
            if (!whole[c]) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see[c] >> k & 1)) x[32 * c + k] = 0.f;
            }
          }
          if constexpr (kKeys) {
            uint32_t p16[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) p16[k] = act[c] ? pack16<T>(x[32 * c + 2 * k], x[32 * c + 2 * k + 1]) : 0u;
            if (h0 < extent) tmem_st16(lanes + kColS + h0 + 16 * c, p16);  // zeros too, to the end of 64 rows
          }
        }
        if constexpr (kKeys) tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
        if (!(ok = mbar_wait_warp(dp_full, m & 1, s_wait))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t d16[16];
          if (act[c]) {
            float y[32];
            tmem_ld32(lanes + kColDP + h0 + 32 * c, reinterpret_cast<uint32_t*>(y));
            tmem_wait_ld32(reinterpret_cast<uint32_t*>(y));
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              float4 de = make_float4(delta, delta, delta, delta);
              if constexpr (kKeys) de = *reinterpret_cast<const float4*>(col + kStream + 32 * c + k);
              const uint64_t p0 = pack2(y[k], y[k + 1]), p1 = pack2(y[k + 2], y[k + 3]);
              const uint64_t d0 = pack2(de.x, de.y), d1 = pack2(de.z, de.w);
              const uint64_t y0 = mul2(kBf16 ? add2(p0, d0) : fma2(p0, c2, d0), pack2(x[32 * c + k], x[32 * c + k + 1]));
              const uint64_t y1 = mul2(kBf16 ? add2(p1, d1) : fma2(p1, c2, d1), pack2(x[32 * c + k + 2], x[32 * c + k + 3]));
              y[k] = lo2(y0);
              y[k + 1] = hi2(y0);
              y[k + 2] = lo2(y1);
              y[k + 3] = hi2(y1);
            }
            if (!whole[c]) {  // 0 times what a hidden pair's dP holds need not be 0
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see[c] >> k & 1)) y[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) d16[k] = pack16<T>(y[2 * k], y[2 * k + 1]);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) d16[k] = 0;
          }
          if (h0 < extent) tmem_st16(lanes + kColDP + h0 + 16 * c, d16);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ds_ready);
      }
      if (!ok) break;
      const bool live = row < w.rows;
      const int64_t at = (((int64_t)w.kept_row + row) * (kKeys ? a.kv_heads : a.heads) + w.h) * a.D;
      float* sums = kKeys && w.slot >= 0
                        ? a.partial + (((int64_t)w.slot * a.kv_heads + w.h) * kTile + row) * (2 * DP)
                        : nullptr;
      const float back = w.back;  // a power of two, as kBackP, so that the products with them are exact
      mbar_arrive(item_empty + 8 * slot);
      if (!kKeys && !(ok = ahead(i + 1))) break;
      const int acc = nk % Sh::kAcc;
      if (!(ok = mbar_wait_warp(acc_full + 8 * acc, (nk / Sh::kAcc) & 1, s_wait))) break;
      tc_fence_after();
      // the parts share the stores: dK and dV, or half of dQ each
      const uint32_t from = lanes + kColAcc + acc * Sh::kAccColumns;
#pragma unroll
      for (int x = part; x < 2; x += Sh::kParts) {
        if (kKeys && sums) {  // a piece of a tile: its float32 sums, to be joined
#pragma unroll 1
          for (int c = 0; c < DP; c += 32) {
            uint32_t v[32];
            tmem_ld32(from + x * DP + c, v);
            tmem_wait_ld32(v);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!kBf16) v[k] = __float_as_uint(__uint_as_float(v[k]) * (x == 0 ? back : Item::kBackP));
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              if (live) *reinterpret_cast<uint4*>(sums + x * DP + c + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        } else if constexpr (kKeys)
          store_row<T, DP>(from + x * DP, live, x == 0 ? a.scale * back : Item::kBackP, static_cast<T*>(x == 0 ? a.d1 : a.d2) + at, a.D,
                           a.sectors);
        else
          store_row<T, DP / 2>(from + x * (DP / 2), live, a.scale * back, static_cast<T*>(a.d1) + at + x * (DP / 2),
                               a.D - x * (DP / 2), a.sectors);
      }
      tc_fence_before();
      mbar_arrive(acc_empty + 8 * acc);
      ++nk;
    }
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

// dK and dV of the key tiles that were cut into pieces: their sums in order.
template <typename T, int DP>
__global__ void __launch_bounds__(256) k_attn_join_keys(const BwdArgs a, const JoinItem* joins) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int slots = a.hdr->n_items[kKeySlots];
  for (int i = blockIdx.x; i < slots * a.kv_heads; i += gridDim.x) {
    const JoinItem j = joins[i / a.kv_heads];
    const int h = i % a.kv_heads;
    if (j.chunks == 0) continue;  // not a tile's first slot
    for (int e = threadIdx.x; e < j.nq * (2 * DP / 4); e += 256) {
      const int row = e / (2 * DP / 4), c = (e - row * (2 * DP / 4)) * 4, d = c % DP;
      if (d >= a.D) continue;
      const float* from = a.partial + (((int64_t)j.slot * a.kv_heads + h) * kTile + row) * (2 * DP) + c;
      const int64_t step = (int64_t)a.kv_heads * kTile * 2 * DP;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = 0; p < j.chunks; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(from + p * step);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
      }
      const float f = c < DP ? a.scale : 1.f;
      T* to = static_cast<T*>(c < DP ? a.d1 : a.d2) + ((int64_t)(j.q0 + row) * a.kv_heads + h) * a.D + d;
      *reinterpret_cast<uint2*>(to) = make_uint2(pack16<T>(s.x * f, s.y * f), pack16<T>(s.z * f, s.w * f));
    }
  }
}

// How a call cuts the key tiles that every query sees: into pieces of so many
// streamed tiles, with so many slots for their sums; 0 where none is long
// enough.  A piece is no shorter than a tile within a window, and than half a
// block's share of the work if it were even.
struct Pieces {
  int piece, slots;
};
Pieces pieces_of(const AttnCall& c) {
  const int64_t stream = c.D <= 64 ? 64 : 128, blocks = 148 * (c.D <= 64 ? 2 : 1);
  const int64_t longest = c.max_tokens > 0 && c.max_tokens < c.n_q ? c.max_tokens : c.n_q;
  const int64_t full = (longest / stream + 2) * c.group, tiles = c.n_kv / kTile + c.B;
  const bool window = c.mask.left < kFar;
  const int64_t sink_tiles = ((int64_t)c.mask.sinks + kTile - 1) / kTile;
  const int64_t in_window = ((int64_t)kTile + c.mask.left + c.mask.right) / stream + 3;
  const int64_t other = window && in_window * c.group < full ? in_window * c.group : full;
  const int64_t long_work = window ? (sink_tiles < tiles ? sink_tiles : tiles) * (c.n_q / stream + 2 * (int64_t)c.B) * c.group
                                   : tiles * full;
  const int64_t work = (window ? tiles * other : 0) + long_work;
  int64_t piece = work * c.kv_heads / (2 * blocks);
  if (piece < 16) piece = 16;
  if (window && piece < other) piece = other;
  if (full <= piece || long_work == 0) return {0, 0};
  return {(int)piece, (int)(2 * long_work / piece + 1)};
}

struct BwdWorkspace {
  WsHeader* hdr;
  TileItem *queries, *keys, *shorts;
  JoinItem* joins;
  float* partial;
  Pieces pieces;
  float *rows, *range;
  size_t bytes;
};
BwdWorkspace carve_backward(void* base, const AttnCall& c) {
  BwdWorkspace w = {};
  const int64_t n_q = c.n_q, n_kv = c.n_kv;
  const int B = c.B, heads = c.heads;
  w.pieces = pieces_of(c);
  char* p = static_cast<char*>(base);
  size_t off = 256;
  const auto take = [&](size_t bytes) {
    char* at = p + off;
    off = (off + bytes + 255) & ~(size_t)255;
    return at;
  };
  w.hdr = reinterpret_cast<WsHeader*>(p);
  w.queries = reinterpret_cast<TileItem*>(take((max_tiles(n_q, B) + 1) * sizeof(TileItem)));
  w.keys = reinterpret_cast<TileItem*>(take((max_tiles(n_kv, B) + w.pieces.slots + 1) * sizeof(TileItem)));
  w.joins = reinterpret_cast<JoinItem*>(take((size_t)w.pieces.slots * sizeof(JoinItem)));
  w.partial = reinterpret_cast<float*>(
      take((size_t)w.pieces.slots * c.kv_heads * kTile * 2 * (c.D <= 64 ? 64 : 128) * sizeof(float)));
  w.shorts = reinterpret_cast<TileItem*>(take((size_t)(B + 1) * sizeof(TileItem)));
  w.rows = reinterpret_cast<float*>(take((size_t)n_q * heads * 2 * sizeof(float)));
  if (c.dtype == FPS_DTYPE_F16) w.range = reinterpret_cast<float*>(take((size_t)n_q * 2 * sizeof(float)));
  w.bytes = off;
  return w;
}

template <typename T, int DP, bool kKeys>
cudaError_t run(const BwdArgs& a, int64_t items, const CUtensorMap& k1, const CUtensorMap& k2, const CUtensorMap& s1,
                const CUtensorMap& s2, cudaStream_t s) {
  using Sh = BwdShape<DP, kKeys>;
  const auto kernel = k_attn_backward<T, DP, kKeys>;
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(kernel), (int)Sh::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t slots = (int64_t)device_info().sm_count * Sh::kBlocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < slots ? items : slots));
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a, k1, k2, s1, s2);
}

template <typename T, int DP>
cudaError_t run_tiles(const AttnCall& c, const BwdWorkspace& ws, const BwdMaps& m, cudaStream_t s) {
  BwdArgs a;
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
  a.rows = ws.rows;
  a.range = ws.range;
  a.hdr = ws.hdr;
  a.test = c.test;
  a.sectors = m.sectors;
  cudaError_t e;
  if (c.n_q > 0) {
    a.d1 = c.dq;
    a.d2 = nullptr;
    a.items = ws.queries;
    if ((e = run<T, DP, false>(a, max_tiles(c.n_q, c.B) * c.heads, m.q, m.d, m.k, m.v, s)) != cudaSuccess) return e;
  }
  if (c.n_kv > 0) {
    a.d1 = c.dk;
    a.d2 = c.dv;
    a.items = ws.keys;
    a.partial = ws.partial;
    if ((e = run<T, DP, true>(a, (max_tiles(c.n_kv, c.B) + ws.pieces.slots) * c.kv_heads, m.k, m.v, m.q, m.d, s)) !=
        cudaSuccess)
      return e;
    if (ws.pieces.slots > 0) {
      const int64_t items = (int64_t)ws.pieces.slots * c.kv_heads, most = (int64_t)device_info().sm_count * 8;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(items < most ? items : most));
      cfg.blockDim = dim3(256);
      cfg.stream = s;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      count_launch();
      if ((e = cudaLaunchKernelEx(&cfg, k_attn_join_keys<T, DP>, a, (const JoinItem*)ws.joins)) != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace

size_t attention_backward_bytes(const AttnCall& c) {
  return carve_backward(nullptr, c).bytes;
}

cudaError_t launch_attention_backward(const AttnCall& c, void* workspace, cudaStream_t s) {
  const BwdWorkspace ws = carve_backward(workspace, c);
  PlanLists lists = {};
  lists.queries = ws.queries;
  lists.keys = ws.keys;
  lists.shorts = ws.shorts;
  lists.of_queries = {{c.dq, nullptr}, (int64_t)c.heads * c.D, nullptr, 0};
  lists.of_keys = {{c.dk, c.dv}, (int64_t)c.kv_heads * c.D, nullptr, 0};
  lists.piece = ws.pieces.piece;
  lists.slots = ws.pieces.slots;
  lists.stream = c.D <= 64 ? 64 : 128;
  lists.key_joins = ws.joins;
  lists.range = ws.range;
  cudaError_t e = launch_attention_plan(c, ws.hdr, lists, s);
  if (e != cudaSuccess || (c.n_q == 0 && c.n_kv == 0)) return e;
  const bool bf16 = c.dtype == FPS_DTYPE_BF16;
  // without queries (or keys) no item has a tile of the other: their maps are not used
  BwdMaps m = {};
  if (c.n_q > 0 && (!attention_map(&m.q, c.q, bf16, c.n_q, c.heads, c.D, c.q_token, c.q_head) ||
                    !attention_map(&m.d, c.dout, bf16, c.n_q, c.heads, c.D, c.do_token, c.do_head)))
    return cudaErrorInvalidValue;
  if (c.n_kv > 0 && (!attention_map(&m.k, c.k, bf16, c.n_kv, c.kv_heads, c.D, c.k_token, c.k_head) ||
                     !attention_map(&m.v, c.v, bf16, c.n_kv, c.kv_heads, c.D, c.v_token, c.v_head)))
    return cudaErrorInvalidValue;
  if (c.n_q == 0) m.q = m.k, m.d = m.v;
  if (c.n_kv == 0) m.k = m.q, m.v = m.d;
  m.sectors = ((reinterpret_cast<uintptr_t>(c.dq) | reinterpret_cast<uintptr_t>(c.dk) | reinterpret_cast<uintptr_t>(c.dv)) &
               31) == 0 &&
              c.D % 16 == 0;
  if (c.n_q > 0 && (e = launch_attention_backward_rows(c, ws.rows, s)) != cudaSuccess) return e;
  if (ws.range && c.n_q > 0 && c.n_kv > 0 &&
      (e = launch_attention_backward_range(c, ws.range, ws.queries, ws.keys, ws.shorts, ws.hdr, s)) != cudaSuccess)
    return e;
  if ((e = launch_attention_backward_short(c, m, ws.rows, ws.range, ws.shorts, ws.hdr, s)) != cudaSuccess) return e;
  if (c.max_tokens > 0 && c.max_tokens <= kTile) return cudaSuccess;  // every event is short
  if (bf16) return c.D <= 64 ? run_tiles<__nv_bfloat16, 64>(c, ws, m, s) : run_tiles<__nv_bfloat16, 128>(c, ws, m, s);
  return c.D <= 64 ? run_tiles<__half, 64>(c, ws, m, s) : run_tiles<__half, 128>(c, ws, m, s);
}

}  // namespace fpstok
