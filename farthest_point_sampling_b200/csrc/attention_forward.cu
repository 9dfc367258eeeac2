// Attention of packed events, forward, on the tensor cores.
//
// One work item is a tile of 128 queries of one event and one head.  With S =
// Q K^T over a tile of 128 keys, the running maximum m and sum l of the
// softmax give
//   P = exp2(c S - c m),  l <- l f + sum P,  O <- O f + P V,  f = exp2(c (m_old - m)),
// c = scale log2(e), and the output is O / l, lse = m scale + ln l.
//
// A block is six warps: one thread loads Q, K and V tiles with TMA, one issues
// the tcgen05 products, and four warps do the softmax with one query row (a
// TMEM lane) per thread, its scores in registers, so that no row crosses
// threads.  S goes to TMEM, P comes back as 16-bit operand A of the second
// product (64-wide heads: beside S, so that the next scores need not wait for
// it; 128-wide: over S, the columns being taken), O stays in TMEM until the
// item ends.  Two blocks share an SM: while one's softmax runs, the other's
// products do.  Blocks are persistent; the loader runs ahead into the next
// items.  Only the 32-key chunks that some of a warp's rows do not see whole
// pay for masks, so one kernel serves every mask (a second one for calls
// without any took 4% longer).
//
// What bounds it: events of a tile or two, memory - 4096 events of up to 128
// tokens, 12 heads of 64: 493 us, 5.6 TB/s; long events, the softmax - 4 causal
// events of 4000 to 9000 tokens, 16 query and 4 key heads of 128: 692 us, 942
// TFLOP/s, where the products alone would take 392 us at the rate of a library's
// large product and the exponentials 280 us; 8 events of 50000 to 200000 tokens
// under a window of 128 on both sides and 16 sinks: 1756 us, of whose scores
// (three key tiles for each query tile, and one of the sinks) a third is masked.
//
// Rounding: P is rounded to the input type for P V; l sums the unrounded
// values.  O is rescaled only when m grows by more than 8 / log2 units, which
// leaves P at most 2^8: exact in the float32 accumulator and far from the
// range limits of both types.
#include <type_traits>

#include "attention_few.h"
#include "attention_plan.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace fpstok {

namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kFwdThreads = kSoftmaxThreads + 64;
constexpr int kPanel = kTile * 128;  // bytes of a 128-row panel of 64 values
constexpr uint32_t kTmemColumns = 256;

struct FwdArgs {
  int64_t n_q;
  int heads, group, D;
  AttnMask mask;
  float scale, scale_log2;
  void* out;
  float* lse;
  const int64_t* q_offsets;
  int B, zero_tail;
  WaitTest test;
  bool sectors;  // every row of out starts on a 32-byte sector, and ends on one
  const TileItem* items;
  WsHeader* hdr;
};

// One work item as the loading thread hands it to the others, through a ring
// in shared memory.
struct FwdItem {
  int count;            // key tiles; -1 ends the work
  int h;                // head
  int q_row, rows, p0;  // first query row, queries of the tile, position of the first
  int k_row, nk;        // the event's first key row, its keys
  KeyTiles<kTile> keys;
};
constexpr int kItemRing = 2;
__device__ __forceinline__ FwdItem fwd_item(const FwdArgs& a, int h, const TileItem& e) {
  FwdItem w;
  w.h = h;
  w.q_row = e.q0 + e.t * kTile;
  w.rows = min(kTile, e.nq - e.t * kTile);
  w.p0 = e.t * kTile + e.nk - e.nq;
  w.k_row = e.k0;
  w.nk = e.nk;
  w.keys = key_tiles<kTile>(a.mask, w.p0, w.p0 + w.rows - 1, e.nk);
  w.count = w.keys.count;
  return w;
}

template <int DP>
struct FwdShape {
  static constexpr int kPanels = DP / 64;
  static constexpr int kStages = DP == 64 ? 2 : 1;  // of Q, K and V each: 96 KB either way, two blocks per SM
  static constexpr uint32_t kTileBytes = kPanels * kPanel;
  // S in columns 0 .. 127; 64-wide heads leave room for P beside it, with
  // 128-wide ones P lies over S and the next S waits for the product that reads it
  static constexpr bool kOver = DP == 128;
  static constexpr uint32_t kColP = kOver ? 0 : 128, kColO = kOver ? 128 : 192;
  static constexpr size_t kSmem =
      1024 + 3 * kStages * kTileBytes + kItemRing * sizeof(FwdItem) + 256;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kFwdThreads, 2)
    k_attn_forward(const FwdArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v) {
  using Sh = FwdShape<DP>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t s_raw[];
  uint8_t* s_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* s_q = s_base;
  uint8_t* s_k = s_q + Sh::kStages * Sh::kTileBytes;
  uint8_t* s_v = s_k + Sh::kStages * Sh::kTileBytes;
  FwdItem* s_item = reinterpret_cast<FwdItem*>(s_v + Sh::kStages * Sh::kTileBytes);
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_item + kItemRing);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_bar + 24);
  volatile WaitState* s_wait = reinterpret_cast<volatile WaitState*>(s_tmem + 1);
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t q_full = bars, k_full = bars + 16, k_empty = bars + 32, v_full = bars + 48, v_empty = bars + 64,
                 s_full = bars + 80, o_full = bars + 88, drain = bars + 96, item_full = bars + 104,
                 item_empty = bars + 120, p_ready = bars + 136, q_empty = bars + 144;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 15; ++i) mbar_init(bars + 8 * i, 1);
    for (int i = 0; i < kItemRing; ++i) mbar_init(item_empty + 8 * i, kSoftmaxThreads + 1);
    mbar_init(p_ready, kSoftmaxThreads);
    for (int i = 0; i < 2; ++i) mbar_init(q_empty + 8 * i, 1);
    s_wait->gave_up = 0;
    s_wait->polls = a.test.polls;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == kSoftmaxWarps + 1) tmem_alloc(smem_u32(s_tmem), kTmemColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*s_tmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == kSoftmaxWarps) {
    // ------------------------------------------------ items and loads
    {
      ItemClaims claims(&a.hdr->next_item[kQueryTiles], a.items, a.heads, a.hdr->n_items[kQueryTiles]);
      // items handed out; tiles of Q, of K and of V whose loads were issued
      int i = 0, n = 0, nq = 0, nv = 0;
      for (bool more = true; more; ++i) {
        const int slot = i % kItemRing;
        if (i >= kItemRing && !mbar_wait_warp(item_empty + 8 * slot, ((i / kItemRing) - 1) & 1, s_wait)) break;
        TileItem entry;
        int h;
        more = claims.take(&entry, &h);
        if (!more) {
          if (lane == 0) s_item[slot].count = -1;
          __syncwarp();
          mbar_arrive_one(item_full + 8 * slot);
          break;
        }
        const FwdItem w = fwd_item(a, h, entry);
        if (lane == 0) s_item[slot] = w;
        __syncwarp();
        mbar_arrive_one(item_full + 8 * slot);
        if (w.count == 0) continue;
        const int qs = nq % Sh::kStages;
        if (nq >= Sh::kStages && !mbar_wait_warp(q_empty + 8 * qs, ((nq / Sh::kStages) - 1) & 1, s_wait)) break;
        const int q_boxes = (w.rows + 63) / 64;
        mbar_expect(q_full + 8 * qs, q_boxes * 8192 * Sh::kPanels);
#pragma unroll 1
        for (int b = 0; b < q_boxes; ++b)
#pragma unroll
          for (int p = 0; p < Sh::kPanels; ++p)
            tma_load(smem_u32(s_q) + qs * Sh::kTileBytes + p * kPanel + b * 8192, &map_q, q_full + 8 * qs, p * 64, w.h,
                     w.q_row + b * 64);
        ++nq;
        const int g = w.h / a.group;
        for (int j = 0; j < w.count; ++j, ++nv) {
          const int st = n % Sh::kStages;
          const uint32_t round = ((n / Sh::kStages) - 1) & 1;
          const int boxes = (w.keys.extent(j) + 63) / 64;
          const int krow = w.k_row + w.keys.start(j);
          if (n >= Sh::kStages && !(more = mbar_wait_warp(k_empty + 8 * st, round, s_wait))) break;
          const bool skip = (a.test.skip & FPS_SKIP_FORWARD) && blockIdx.x == 0 && n == 0;
          if (!skip) mbar_expect(k_full + 8 * st, boxes * 8192 * Sh::kPanels);
#pragma unroll 1
          for (int b = 0; b < (skip ? 0 : boxes); ++b)
#pragma unroll
            for (int p = 0; p < Sh::kPanels; ++p)
              tma_load(smem_u32(s_k) + st * Sh::kTileBytes + p * kPanel + b * 8192, &map_k, k_full + 8 * st, p * 64, g,
                       krow + b * 64);
          ++n;
          if (nv >= Sh::kStages && !(more = mbar_wait_warp(v_empty + 8 * st, round, s_wait))) break;
          mbar_expect(v_full + 8 * st, boxes * 8192 * Sh::kPanels);
#pragma unroll 1
          for (int b = 0; b < boxes; ++b)
#pragma unroll
            for (int p = 0; p < Sh::kPanels; ++p)
              tma_load(smem_u32(s_v) + st * Sh::kTileBytes + p * kPanel + b * 8192, &map_v, v_full + 8 * st, p * 64, g,
                       krow + b * 64);
        }
      }
      // after a wait that gave up: the copies still in flight land first, at most
      // the last one of each stage
      if (__any_sync(kFull, s_wait->gave_up)) {
        for (int b = 1; b <= Sh::kStages; ++b) {
          if (nq >= b) mbar_land_warp(q_full + 8 * ((nq - b) % Sh::kStages), ((nq - b) / Sh::kStages) & 1, s_wait);
          if (n >= b) mbar_land_warp(k_full + 8 * ((n - b) % Sh::kStages), ((n - b) / Sh::kStages) & 1, s_wait);
          if (nv >= b) mbar_land_warp(v_full + 8 * ((nv - b) % Sh::kStages), ((nv - b) / Sh::kStages) & 1, s_wait);
        }
      }
    }
  } else if (warp == kSoftmaxWarps + 1) {
    // ------------------------------------------------ products
    {
      int n = 0, nq = 0;
      const uint32_t pv_desc = mma_desc(kBf16, false, true, (a.D + 15) / 16 * 16);
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int slot = i % kItemRing;
        if (!(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) break;
        const int count = uniform(s_item[slot].count);
        KeyTiles<kTile> keys;
        keys.before = uniform(s_item[slot].keys.before);
        keys.first = uniform(s_item[slot].keys.first);
        keys.end = uniform(s_item[slot].keys.end);
        keys.s = uniform(s_item[slot].keys.s);
        mbar_arrive_one(item_empty + 8 * slot);
        if (count < 0) break;
        if (count == 0) continue;
        const int qs = nq % Sh::kStages;
        const uint32_t q = smem_desc(smem_u32(s_q) + qs * Sh::kTileBytes, kPanel);
        if (!(ok = mbar_wait_warp(q_full + 8 * qs, (nq / Sh::kStages) & 1, s_wait))) break;
        for (int j = 0; j <= count; ++j) {
          if (j > 0) {  // O += P V of tile j - 1
            const int m = n + j - 1, st = m % Sh::kStages;
            const bool both = keys.extent(j - 1) > 64;
            if (!(ok = mbar_wait_warp(v_full + 8 * st, (m / Sh::kStages) & 1, s_wait))) break;
            if (!(ok = mbar_wait_warp(p_ready, m & 1, s_wait))) break;
            tc_fence_after();
            const uint32_t v = smem_desc(smem_u32(s_v) + st * Sh::kTileBytes, kPanel);
            mma_ts(tmem + Sh::kColO, tmem + Sh::kColP, v, pv_desc, j > 1);
            if (both) mma_ts(tmem + Sh::kColO, tmem + Sh::kColP + 32, v + kRun, pv_desc, true);
            mma_commit(v_empty + 8 * st);
            if (j == count) mma_commit(o_full);
            // products of different shapes are not promised to run in order
            if (Sh::kOver && !(ok = mbar_wait_warp(v_empty + 8 * st, (m / Sh::kStages) & 1, s_wait))) break;
          }
          if (j < count) {  // S = Q K^T of tile j
            const int m = n + j, st = m % Sh::kStages;
            const int cols = (keys.extent(j) + 15) / 16 * 16;
            if (!(ok = mbar_wait_warp(k_full + 8 * st, (m / Sh::kStages) & 1, s_wait))) break;
            tc_fence_after();
            const uint32_t k = smem_desc(smem_u32(s_k) + st * Sh::kTileBytes, kPanel);
            const uint32_t qk_desc = mma_desc(kBf16, false, false, cols);
            // whole panels: values past D are zeros
#pragma unroll
            for (int p = 0; p < Sh::kPanels; ++p) mma_ss<2, 2>(tmem, q + p * (kPanel >> 4), k + p * (kPanel >> 4), qk_desc, p > 0);
            mma_commit(k_empty + 8 * st);
            mma_commit(s_full);
            if (j == count - 1) mma_commit(q_empty + 8 * qs);
          }
        }
        n += count;
        ++nq;
      }
      if (__any_sync(kFull, s_wait->gave_up)) {  // products in flight end before TMEM is freed
        mma_commit(drain);
        mbar_land_warp(drain, 0, s_wait);
      }
    }
  } else {
    // ------------------------------------------------ softmax
    int n = 0, nq = 0;  // key tiles and query tiles so far
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int slot = i % kItemRing;
      if (!(ok = mbar_wait_warp(item_full + 8 * slot, (i / kItemRing) & 1, s_wait))) break;
      const FwdItem& w = s_item[slot];  // read where it is needed: it stays until this thread lets go of the slot
      const int count = w.count;
      if (count < 0) break;
      const int warp_rows = min(32, w.rows - warp * 32);
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < count; ++j, ++n) {
        const int k0 = w.keys.start(j), extent = w.keys.extent(j);
        // the tile's 32-key chunks, one lane each: which of them some row of the
        // warp sees, and of which all its rows see every key
        constexpr int kChunks = kTile / 32;
        const int pa = w.p0 + warp * 32;
        const int pb = pa + warp_rows - 1, key = k0 + 32 * lane;
        const bool some = 32 * lane < extent && warp_rows > 0 && some_seen(a.mask, pa, pb, key);
        const bool all = 32 * lane + 32 <= extent && all_seen(a.mask, pa, pb, key);
        const uint32_t act = __ballot_sync(kFull, some && lane < kChunks), whole = __ballot_sync(kFull, all);
        if (!(ok = mbar_wait_warp(s_full, n & 1, s_wait))) break;
        tc_fence_after();
        // Only now is the values' barrier waited for: with one stage, before these
        // scores it may still be in the phase of the tile before, whose end looks
        // the same as that of the tile before it.
        const int left = w.nk - k0;
        if (rows_to_clear(extent, left)) {
          const int st = n % Sh::kStages;
          if (!(ok = mbar_wait_warp(v_full + 8 * st, (n / Sh::kStages) & 1, s_wait))) break;
          clear_rows<Sh::kPanels>(s_v + st * Sh::kTileBytes, extent, left, threadIdx.x, kSoftmaxThreads);
          fence_async_smem();
        }
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tmem_ld32(lanes + 32 * c, reinterpret_cast<uint32_t*>(s + 32 * c));
#pragma unroll
        for (int c = 0; c < kChunks; ++c) tmem_wait_ld32(reinterpret_cast<uint32_t*>(s + 32 * c));
        if (act & ~whole) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (act >> c & ~whole >> c & 1) {  // what this row sees of it
              const uint32_t see = bits(0, extent - 32 * c) & seen_keys(a.mask, pa + lane, k0 + 32 * c);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(see >> k & 1)) s[32 * c + k] = -INFINITY;
            }
        }
        float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (act >> c & 1) {
#pragma unroll
            for (int k = 32 * c; k < 32 * c + 32; k += 8) {
              m0 = max3f(m0, s[k], s[k + 1]);
              m1 = max3f(m1, s[k + 2], s[k + 3]);
              m2 = max3f(m2, s[k + 4], s[k + 5]);
              m3 = max3f(m3, s[k + 6], s[k + 7]);
            }
          }
        const float top = fmaxf(max3f(m0, m1, m2), m3);
        if (j == 0) {
          m_used = top;
        } else {
          // a row that has seen nothing yet takes its first maximum at once
          const bool grow = top > m_used && (m_used == -INFINITY || (top - m_used) * a.scale_log2 > 8.f);
          if (__any_sync(kFull, grow)) {
            const float f = !grow ? 1.f : m_used == -INFINITY ? 0.f : exp2_approx((m_used - top) * a.scale_log2);
            if (grow) m_used = top;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP; c += 8) {
              uint32_t o[8];
              tmem_ld8(lanes + Sh::kColO + c, o);
              tmem_wait_ld8(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st8(lanes + Sh::kColO + c, o);
            }
          }
        }
        const float base = m_used == -INFINITY ? 0.f : m_used * a.scale_log2;
        const float2 base2 = make_float2(-base, -base), scale2 = make_float2(a.scale_log2, a.scale_log2);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t pk[16];
          if (act >> c & 1) {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float2 e = fma2(make_float2(s[32 * c + k], s[32 * c + k + 1]), scale2, base2);
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              sum = add2(sum, e);
              pk[k / 2] = pack16<T>(e.x, e.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[k] = 0;
          }
          if (32 * (c & ~1) < extent) tmem_st16(lanes + Sh::kColP + 16 * c, pk);  // zeros too, to the end of 64 keys
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
      }
      if (!ok) break;
      const int64_t first_row = (int64_t)w.q_row + warp * 32;
      T* out = static_cast<T*>(a.out) + (first_row * a.heads + w.h) * a.D;
      float* lse = a.lse ? a.lse + (int64_t)w.h * a.n_q + first_row : nullptr;
      const int64_t row_values = (int64_t)a.heads * a.D;
      mbar_arrive(item_empty + 8 * slot);
      if (count == 0) {  // nothing to see
        if (lane < warp_rows) {
#pragma unroll 1
          for (int c = 0; c < a.D; c += 8)
            *reinterpret_cast<uint4*>(out + lane * row_values + c) = make_uint4(0, 0, 0, 0);
          if (lse) lse[lane] = -INFINITY;
        }
        continue;
      }
      if (!(ok = mbar_wait_warp(o_full, nq & 1, s_wait))) break;
      ++nq;
      tc_fence_after();
      // O / l.  Where a row saw no key O may hold what masked infinities left, so
      // such rows are cleared, not scaled.
      const bool live = lane < warp_rows;
      if (__any_sync(kFull, l == 0.f)) {
#pragma unroll 1
        for (int c = 0; c < DP; c += 8) {
          uint32_t o[8];
          tmem_ld8(lanes + Sh::kColO + c, o);
          tmem_wait_ld8(o);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = l == 0.f ? 0u : o[k];
          tmem_st8(lanes + Sh::kColO + c, o);
        }
        tmem_wait_st();
      }
      store_row<T, DP>(lanes + Sh::kColO, live, l == 0.f ? 0.f : rcp_approx(l), out + lane * row_values, a.D, a.sectors);
      tc_fence_before();
      if (lse && live) lse[lane] = l == 0.f ? -INFINITY : fmaf(m_used, a.scale, log2_approx(l) * kLn2);
    }
  }
  if (a.zero_tail && rows_known(a.hdr))
    clear_tail(a.zero_tail, a.out, a.lse, a.B > 0 ? a.q_offsets[a.B] : 0, a.n_q, a.heads, a.D);
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
  if (threadIdx.x == 0 && s_wait->gave_up) record_error(a.hdr, kDevWaitTimeout);
}

// Whether a call looks for events with at most kFewRows query rows: when its
// events have no more than that on average.  One query for each of 8 events of
// 50000 to 200000 tokens, 12 and 4 heads of 64: 206 us, and 2503 us in tiles of
// 128 queries by this kernel; one event of 128 tokens takes 14 us either way.
bool few_rows(const AttnCall& c) { return c.B > 0 && c.n_q * c.group <= (int64_t)kFewRows * c.B; }

struct FwdWorkspace {
  WsHeader* hdr;
  TileItem* items;
  TileItem* units;
  JoinItem* joins;
  float* partial;
  int chunk;
  size_t bytes;
};
FwdWorkspace carve_forward(void* base, const AttnCall& c) {
  FwdWorkspace w = {};
  char* p = static_cast<char*>(base);
  size_t off = 256;
  const auto take = [&](size_t bytes) {
    char* at = p + off;
    off = (off + bytes + 255) & ~(size_t)255;
    return at;
  };
  w.hdr = reinterpret_cast<WsHeader*>(p);
  w.items = reinterpret_cast<TileItem*>(take((max_tiles(c.n_q, c.B) + 1) * sizeof(TileItem)));
  if (few_rows(c)) {
    w.chunk = few_chunk(c.n_kv, c.kv_heads);
    w.units = reinterpret_cast<TileItem*>(take((c.n_kv / w.chunk + c.B + 1) * sizeof(TileItem)));
    w.joins = reinterpret_cast<JoinItem*>(take((c.n_kv / w.chunk + 1) * sizeof(JoinItem)));
    w.partial = reinterpret_cast<float*>(take(few_partial_floats(c.n_kv, c.kv_heads, c.D, w.chunk) * sizeof(float)));
  }
  w.bytes = off;
  return w;
}

template <typename T, int DP>
cudaError_t run_forward(const AttnCall& c, const FwdWorkspace& ws, cudaStream_t s) {
  cudaError_t e;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  CUtensorMap map_q, map_k, map_v;
  if (!attention_map(&map_q, c.q, bf16, c.n_q, c.heads, c.D, c.q_token, c.q_head)) return cudaErrorInvalidValue;
  map_k = map_v = map_q;  // without keys no item has a key tile: the maps are not used
  if (c.n_kv > 0 && (!attention_map(&map_k, c.k, bf16, c.n_kv, c.kv_heads, c.D, c.k_token, c.k_head) ||
                     !attention_map(&map_v, c.v, bf16, c.n_kv, c.kv_heads, c.D, c.v_token, c.v_head)))
    return cudaErrorInvalidValue;
  FwdArgs a;
  a.n_q = c.n_q;
  a.heads = c.heads;
  a.group = c.group;
  a.D = c.D;
  a.mask = c.mask;
  a.scale = c.scale;
  a.scale_log2 = c.scale * kLog2e;
  a.out = c.out;
  a.lse = c.lse;
  a.q_offsets = c.q_offsets;
  a.B = c.B;
  a.zero_tail = few_rows(c) ? 0 : c.zero_tail;  // the other kernel has done it
  a.sectors = reinterpret_cast<uintptr_t>(c.out) % 32 == 0 && c.D % 16 == 0;
  a.test = c.test;
  a.items = ws.items;
  a.hdr = ws.hdr;
  const auto kernel = k_attn_forward<T, DP>;
  constexpr int smem = (int)FwdShape<DP>::kSmem;
  e = allow_shared_memory(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t items = max_tiles(c.n_q, c.B) * c.heads;
  const int64_t slots = (int64_t)device_info().sm_count * 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < slots ? items : slots));
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a, map_q, map_k, map_v);
}

template <typename T>
cudaError_t run_type(const AttnCall& c, const FwdWorkspace& ws, cudaStream_t s) {
  return c.D <= 64 ? run_forward<T, 64>(c, ws, s) : run_forward<T, 128>(c, ws, s);
}

}  // namespace

size_t attention_forward_bytes(const AttnCall& c) { return carve_forward(nullptr, c).bytes; }

cudaError_t launch_attention_forward(const AttnCall& c, void* workspace, cudaStream_t s) {
  const FwdWorkspace ws = carve_forward(workspace, c);
  PlanLists lists = {};
  lists.queries = ws.items;
  lists.of_queries = {{c.out, nullptr}, (int64_t)c.heads * c.D, c.lse, c.heads};
  if (few_rows(c)) {
    lists.units = ws.units;
    lists.joins = ws.joins;
    lists.chunk = ws.chunk;
  }
  cudaError_t e = launch_attention_plan(c, ws.hdr, lists, s);
  if (e != cudaSuccess || c.n_q == 0) return e;
  if (lists.units) {
    const FewPlan plan = {ws.chunk, ws.units, ws.joins, ws.partial};
    if ((e = launch_attention_few(c, plan, ws.hdr, s)) != cudaSuccess) return e;
    if (c.n_q * c.group <= kFewRows) return cudaSuccess;  // no event can have more rows than the call
  }
  return c.dtype == FPS_DTYPE_BF16 ? run_type<__nv_bfloat16>(c, ws, s) : run_type<__half>(c, ws, s);
}

}  // namespace fpstok
