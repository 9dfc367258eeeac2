// Attention of packed events, backward, on the tensor cores.
//
// With S, P and lse of the forward and D_i = sum_d dO_id O_id,
//   dV = P^T dO,   dP = dO V^T,   dS = P (dP - D),   dQ = scale dS K,   dK = scale dS^T Q,
// the K and V gradients summed over the query heads that share them.
//
// Two kernels, one template.  A work item keeps a 128-row tile of one pair of
// tensors and streams 64-row tiles of the other past it:
//   queries: keeps Q, dO of one query tile and head, streams K, V:
//            scores S = Q K^T and dP = dO V^T, then dQ += dS K;
//   keys:    keeps K, V of one key tile and key head, streams Q, dO of every
//            query tile that sees it, for every head of the group:
//            S^T = K Q^T and dP^T = V dO^T, then dV += P^T dO, dK += dS^T Q.
// P is formed again from the scores and lse.  Each gradient tile is summed by
// one block in a fixed order, so the result does not depend on scheduling;
// the price is that the scores are formed twice.
//
// Roles as in the forward kernel: a loading thread, an issuing thread, and
// softmax warps with one kept row per thread; P and dS go back to TMEM as
// 16-bit operand A.  TMEM holds kGroups stages of scores (128 columns each)
// and the accumulators.  With 64-wide heads a block takes 256 columns and two
// blocks share an SM; with 128-wide heads the keys kernel takes all 512 and
// works on two stages at once with a warp group each.
//
// Rounding: P and dS are rounded to the input type for their products.  D
// comes from the rounded output, as the forward left it.
#include <type_traits>

#include "attention_plan.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace fpstok {

namespace {

constexpr int kStream = 64;                   // rows of a streamed tile
constexpr int kStreamPanel = kStream * 128;   // bytes of one of its 64-value panels
constexpr int kPanel = kTile * 128;

struct BwdArgs {
  int64_t n_q, n_kv;
  int heads, kv_heads, group, D;
  AttnMask mask;
  float scale, scale_log2;
  const void* out;
  const float* lse;
  float* delta;  // [heads, n_q], written by the queries kernel
  void* d1;      // dQ, or dK
  void* d2;      // dV
  const int64_t* offsets;  // of the kept rows
  int B;
  bool sectors;  // every gradient row starts on a 32-byte sector, and ends on one
  const TileItem* items;
  WsHeader* hdr;
};

template <int DP, int kGroups, bool kKeys>
struct BwdShape {
  static constexpr int kPanels = DP / 64;
  static constexpr uint32_t kKeptBytes = kPanels * kPanel;          // one kept tensor's tile
  static constexpr uint32_t kStreamBytes = kPanels * kStreamPanel;  // one streamed tensor's tile
  // 96 KB and two blocks per SM, or 192 KB and one
  static constexpr int kKept = DP == 64 || kKeys ? 2 : 1;
  static constexpr int kRing = DP == 64 || kKeys ? 2 : 1;
  static constexpr int kThreads = 32 * (4 * kGroups + 2);
  static constexpr uint32_t kColAcc = 128 * kGroups;
  static constexpr uint32_t kColumns = kColAcc + (kKeys ? 2 : 1) * DP <= 256 ? 256 : 512;
  static constexpr int kBlocks = kColumns == 256 ? 2 : 1;
  static constexpr size_t kSmem = 1024 + 2 * (kKept * kKeptBytes + kRing * kStreamBytes) + kGroups * 1024 + 256;
};

struct BwdItem {
  TileItem e;
  int h;           // head (queries kernel) or key head
  int row0, rows;  // kept rows: first in its event, how many
  int shift;       // nk - nq: position of query 0
  KeyTiles<kStream> tiles;  // streamed tiles of one head
  int count;       // streamed tiles in all
};
template <bool kKeys>
__device__ __forceinline__ BwdItem bwd_item(const BwdArgs& a, int h, const TileItem& e) {
  BwdItem w;
  w.h = h;
  w.e = e;
  w.row0 = w.e.t * kTile;
  w.rows = min(kTile, (kKeys ? w.e.nk : w.e.nq) - w.row0);
  w.shift = w.e.nk - w.e.nq;
  if constexpr (kKeys) {
    // queries that see some key of the tile: the first key's lower and the
    // last key's upper bound; a tile with a sink in it is seen to the end
    const ColumnSpan first = column_span(a.mask, w.row0), last = column_span(a.mask, w.row0 + w.rows - 1);
    const int lo = min(max(first.lo - w.shift, 0), w.e.nq);
    const int hi = min(max(max(first.hi, last.hi) - w.shift + 1, 0), w.e.nq);
    w.tiles.before = w.tiles.s = 0;
    w.tiles.first = lo & ~15;
    w.tiles.end = hi;
    w.tiles.count = hi > lo ? (hi - w.tiles.first + kStream - 1) / kStream : 0;
    w.count = w.tiles.count * a.group;
  } else {
    w.tiles = key_tiles<kStream>(a.mask, w.row0 + w.shift, w.row0 + w.rows - 1 + w.shift, w.e.nk);
    w.count = w.tiles.count;
  }
  return w;
}

// Streamed tile t of an item: the head its rows belong to, first row in the event, rows.
struct StreamTile {
  int head, row0, rows;
};
template <bool kKeys>
__device__ __forceinline__ StreamTile stream_tile(const BwdArgs& a, const BwdItem& w, int t) {
  StreamTile s;
  if constexpr (kKeys) {
    const int m = t / w.tiles.count;
    s.head = w.h * a.group + m;
    s.row0 = w.tiles.start(t - m * w.tiles.count);
    s.rows = w.tiles.extent(t - m * w.tiles.count);
  } else {
    s.head = w.h / a.group;
    s.row0 = w.tiles.start(t);
    s.rows = w.tiles.extent(t);
  }
  return s;
}

template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// One gradient row from its accumulator, or zeros where no tile was seen.
template <typename T, int DP>
__device__ __forceinline__ void gradient_row(uint32_t acc, bool filled, bool live, float f, T* to, int D, bool sectors) {
  if (filled) {
    store_row<T, DP>(acc, live, f, to, D, sectors);
  } else if (live) {
#pragma unroll 1
    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(to + c) = make_uint4(0, 0, 0, 0);
  }
}

template <typename T, int DP, int kGroups, bool kKeys>
__global__ void __launch_bounds__(BwdShape<DP, kGroups, kKeys>::kThreads, BwdShape<DP, kGroups, kKeys>::kBlocks)
    k_attn_backward(const BwdArgs a, const __grid_constant__ CUtensorMap map_k1, const __grid_constant__ CUtensorMap map_k2,
                    const __grid_constant__ CUtensorMap map_s1, const __grid_constant__ CUtensorMap map_s2) {
  using Sh = BwdShape<DP, kGroups, kKeys>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kLoadWarp = 4 * kGroups, kMmaWarp = kLoadWarp + 1;
  extern __shared__ uint8_t s_raw[];
  uint8_t* s_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  // kept tiles (tensor 1 and 2 of a stage side by side), then the streamed ring
  uint8_t* s_kept = s_base;
  uint8_t* s_ring = s_kept + 2 * Sh::kKept * Sh::kKeptBytes;
  float* s_col = reinterpret_cast<float*>(s_ring + 2 * Sh::kRing * Sh::kStreamBytes);  // [group][2][lse, D][64]
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_col + kGroups * 256);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_bar + 18);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t kept_full = bars, kept_empty = bars + 16, ring_full = bars + 32, ring_empty = bars + 48,
                 score_full = bars + 64, ready = bars + 80, acc_full = bars + 96, acc_empty = bars + 104,
                 drain = bars + 112, col_ready = bars + 120;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 10; ++i) mbar_init(bars + 8 * i, 1);
    mbar_init(ready, 128);
    mbar_init(ready + 8, 128);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 128 * kGroups);
    mbar_init(drain, 1);
    mbar_init(col_ready, 128);
    mbar_init(col_ready + 8, 128);
    *s_abort = 0;
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
  const uint32_t tmem = *s_tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // every role walks the block's items, and reads the next one's entry while it works on one
  ItemWalk walk(kKeys ? a.kv_heads : a.heads, a.hdr->n_items[kKeys ? kKeyTiles : kQueryTiles]);
  TileItem next = a.items[walk.more() ? walk.tile : 0];

  if (warp == kLoadWarp) {
    // ------------------------------------------------ loads
    if (lane == 0) {
      int n = 0, nk = 0;  // streamed and kept tiles loaded so far
      bool ok = true;
      while (walk.more() && ok) {
        const BwdItem w = bwd_item<kKeys>(a, walk.h, next);
        walk.advance();
        if (walk.more()) next = a.items[walk.tile];
        if (w.count == 0) continue;
        const int ks = nk % Sh::kKept;
        if (nk >= Sh::kKept && !(ok = mbar_wait(kept_empty + 8 * ks, ((nk / Sh::kKept) - 1) & 1, s_abort))) break;
        const int boxes = (w.rows + 63) / 64;
        const int row = (kKeys ? w.e.k0 : w.e.q0) + w.row0;
        mbar_expect(kept_full + 8 * ks, 2 * boxes * 8192 * Sh::kPanels);
        for (int p = 0; p < Sh::kPanels; ++p)
          for (int i = 0; i < boxes; ++i) {
            const uint32_t to = smem_u32(s_kept) + 2 * ks * Sh::kKeptBytes + p * kPanel + i * 8192;
            tma_load(to, &map_k1, kept_full + 8 * ks, p * 64, w.h, row + i * 64);
            tma_load(to + Sh::kKeptBytes, &map_k2, kept_full + 8 * ks, p * 64, w.h, row + i * 64);
          }
        ++nk;
        for (int t = 0; t < w.count; ++t, ++n) {
          const StreamTile s = stream_tile<kKeys>(a, w, t);
          const int st = n % Sh::kRing;
          if (n >= Sh::kRing && !(ok = mbar_wait(ring_empty + 8 * st, ((n / Sh::kRing) - 1) & 1, s_abort))) break;
          const int srow = (kKeys ? w.e.q0 : w.e.k0) + s.row0;
          mbar_expect(ring_full + 8 * st, 2 * Sh::kStreamBytes);
          for (int p = 0; p < Sh::kPanels; ++p) {
            const uint32_t to = smem_u32(s_ring) + 2 * st * Sh::kStreamBytes + p * kStreamPanel;
            tma_load(to, &map_s1, ring_full + 8 * st, p * 64, s.head, srow);
            tma_load(to + Sh::kStreamBytes, &map_s2, ring_full + 8 * st, p * 64, s.head, srow);
          }
        }
      }
      // after a wait that gave up: this thread's copies still in flight land first
      if (*s_abort) {
        volatile int none = 0;
        for (int i = 0; i < 2; ++i) {
          const int lk = nk - 1 - i, ls = n - 1 - i;
          if (lk >= 0 && i < Sh::kKept) mbar_wait(kept_full + 8 * (lk % Sh::kKept), (lk / Sh::kKept) & 1, &none);
          if (ls >= 0 && i < Sh::kRing) mbar_wait(ring_full + 8 * (ls % Sh::kRing), (ls / Sh::kRing) & 1, &none);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ products
    if (lane == 0) {
      int n = 0, nk = 0;
      const int d_steps = (a.D + 15) / 16;
      const uint32_t out_desc = mma_desc(kBf16, false, true, d_steps * 16);
      bool ok = true;
      while (walk.more() && ok) {
        const BwdItem w = bwd_item<kKeys>(a, walk.h, next);
        walk.advance();
        if (walk.more()) next = a.items[walk.tile];
        if (w.count == 0) continue;
        const int ks = nk % Sh::kKept;
        const uint32_t kept = smem_desc(smem_u32(s_kept) + 2 * ks * Sh::kKeptBytes, kPanel);
        if (!(ok = mbar_wait(kept_full + 8 * ks, (nk / Sh::kKept) & 1, s_abort))) break;
        for (int t = 0; t < w.count + kGroups - 1; ++t) {
          if (t < w.count) {  // scores of tile t, over the P and dS that the products before have read
            const int m = n + t, st = m % Sh::kRing, g = m % kGroups;
            const uint32_t ring = smem_u32(s_ring) + 2 * st * Sh::kStreamBytes;
            const int cols = (stream_tile<kKeys>(a, w, t).rows + 15) / 16 * 16;
            if (!(ok = mbar_wait(ring_full + 8 * st, (m / Sh::kRing) & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t desc = mma_desc(kBf16, false, false, cols);
            const uint32_t from = smem_desc(ring, kStreamPanel);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int k = 0; k < DP / 16; ++k)
                if (k < d_steps)
                  mma_ss(tmem + g * 128 + x * 64,
                         kept + ((x * Sh::kKeptBytes + (k >> 2) * kPanel + (k & 3) * 32) >> 4),
                         from + ((x * Sh::kStreamBytes + (k >> 2) * kStreamPanel + (k & 3) * 32) >> 4), desc, k > 0);
            mma_commit(score_full + 8 * g);
          }
          const int u = t - (kGroups - 1);
          if (u >= 0) {  // gradients from tile u
            const int m = n + u, st = m % Sh::kRing, g = m % kGroups;
            const uint32_t ring = smem_u32(s_ring) + 2 * st * Sh::kStreamBytes;
            const int steps = (stream_tile<kKeys>(a, w, u).rows + 15) / 16;
            if (u == 0 && nk > 0 && !(ok = mbar_wait(acc_empty, (nk - 1) & 1, s_abort))) break;
            if (!(ok = mbar_wait(ready + 8 * g, (m / kGroups) & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t from = smem_desc(ring, kStreamPanel);
            if constexpr (kKeys) {  // dV += P^T dO
#pragma unroll
              for (int k = 0; k < kStream / 16; ++k)
                if (k < steps)
                  mma_ts(tmem + Sh::kColAcc + DP, tmem + g * 128 + k * 8, from + (Sh::kStreamBytes >> 4) + k * 128,
                         out_desc, k > 0 || u > 0);
            }
#pragma unroll
            for (int k = 0; k < kStream / 16; ++k)  // dK += dS^T Q, or dQ += dS K
              if (k < steps)
                mma_ts(tmem + Sh::kColAcc, tmem + g * 128 + 64 + k * 8, from + k * 128, out_desc, k > 0 || u > 0);
            mma_commit(ring_empty + 8 * st);
            if (u == w.count - 1) {
              mma_commit(kept_empty + 8 * ks);
              mma_commit(acc_full);
            }
          }
        }
        if (!ok) break;
        n += w.count;
        ++nk;
      }
      if (*s_abort) {  // products in flight end before TMEM is freed
        volatile int none = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &none);
      }
    }
  } else {
    // ------------------------------------------------ softmax and its gradient
    const int g = warp >> 2;  // warp group: takes the tiles of its score stage
    const int row = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scores = lanes + g * 128;
    float* col = s_col + g * 256;
    int n = 0, nk = 0;
    bool ok = true;
    while (walk.more() && ok) {
      const BwdItem w = bwd_item<kKeys>(a, walk.h, next);
      walk.advance();
      if (walk.more()) next = a.items[walk.tile];
      const bool live = row < w.rows;
      ColumnSpan cs = {0, 0};
      float lse2 = 0.f, delta = 0.f;
      if constexpr (kKeys) {
        cs = column_span(a.mask, w.row0 + row);
      } else if (w.count) {
        // D of this thread's query: dO from its tile, O from memory
        const int ks = nk % Sh::kKept;
        if (!(ok = mbar_wait(kept_full + 8 * ks, (nk / Sh::kKept) & 1, s_abort))) break;
        if (live) {
          const int64_t q = (int64_t)w.e.q0 + w.row0 + row;
          const T* o = static_cast<const T*>(a.out) + (q * a.heads + w.h) * a.D;
          const uint8_t* d = s_kept + (2 * ks + 1) * Sh::kKeptBytes + row * 128;
          for (int c = 0; c < a.D / 8; ++c) {
            const uint4 vo = *reinterpret_cast<const uint4*>(o + c * 8);
            const uint4 vd = *reinterpret_cast<const uint4*>(d + (c >> 3) * kPanel + (((c & 7) ^ (row & 7)) << 4));
            const uint32_t* po = reinterpret_cast<const uint32_t*>(&vo);
            const uint32_t* pd = reinterpret_cast<const uint32_t*>(&vd);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = unpack16<T>(po[i]), y = unpack16<T>(pd[i]);
              delta = fmaf(x.x, y.x, fmaf(x.y, y.y, delta));
            }
          }
          lse2 = a.lse[(int64_t)w.h * a.n_q + q] * kLog2e;
          a.delta[(int64_t)w.h * a.n_q + q] = delta;
        }
      }
      for (int t = 0; t < w.count; ++t) {
        const int m = n + t;
        if (m % kGroups != g) continue;
        const StreamTile s = stream_tile<kKeys>(a, w, t);
        const int visit = m / kGroups;
        const float* c_lse = col + (visit & 1) * 128;
        if constexpr (kKeys) {
          // lse and D of the tile's queries, shared by the rows; one array
          // per parity, so one barrier per tile is enough
          const int64_t at = (int64_t)s.head * a.n_q + w.e.q0 + s.row0 + (row & 63);
          float v = 0.f;
          if ((row & 63) < s.rows) v = row < 64 ? a.lse[at] * kLog2e : a.delta[at];
          col[(visit & 1) * 128 + row] = v;
          mbar_arrive(col_ready + 8 * g);
          if (!(ok = mbar_wait(col_ready + 8 * g, visit & 1, s_abort))) break;
        }
        const int odd = s.rows & 15;
        if (odd) {
          // Streamed rows past the event's last inside a product's step of 16:
          // their P and dS are 0, and the rows must be finite for 0 to stay 0.
          const int st = m % Sh::kRing;
          if (!(ok = mbar_wait(ring_full + 8 * st, (m / Sh::kRing) & 1, s_abort))) break;
          uint8_t* tile = s_ring + 2 * st * Sh::kStreamBytes;
          constexpr int kTensors = kKeys ? 2 : 1;
          for (int e = row; e < (16 - odd) * 8 * Sh::kPanels * kTensors; e += 128) {
            const int c = e % (8 * Sh::kPanels * kTensors), r = s.rows + e / (8 * Sh::kPanels * kTensors);
            *reinterpret_cast<uint4*>(tile + (c >> 3) * kStreamPanel + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        if (!(ok = mbar_wait(score_full + 8 * g, visit & 1, s_abort))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kStream; c += 32) {
          if (c >= s.rows) break;
          float x[32], y[32];
          tmem_ld32(scores + c, reinterpret_cast<uint32_t*>(x));
          tmem_ld32(scores + 64 + c, reinterpret_cast<uint32_t*>(y));
          tmem_wait_ld32(reinterpret_cast<uint32_t*>(x));
          tmem_wait_ld32(reinterpret_cast<uint32_t*>(y));
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float4 le, de;
            if constexpr (kKeys) {
              le = *reinterpret_cast<const float4*>(c_lse + c + i);
              de = *reinterpret_cast<const float4*>(c_lse + 64 + c + i);
            } else {
              le = make_float4(lse2, lse2, lse2, lse2);
              de = make_float4(delta, delta, delta, delta);
            }
            x[i] = exp2_approx(fmaf(x[i], a.scale_log2, -le.x));
            x[i + 1] = exp2_approx(fmaf(x[i + 1], a.scale_log2, -le.y));
            x[i + 2] = exp2_approx(fmaf(x[i + 2], a.scale_log2, -le.z));
            x[i + 3] = exp2_approx(fmaf(x[i + 3], a.scale_log2, -le.w));
            y[i] = x[i] * (y[i] - de.x);
            y[i + 1] = x[i + 1] * (y[i + 1] - de.y);
            y[i + 2] = x[i + 2] * (y[i + 2] - de.z);
            y[i + 3] = x[i + 3] * (y[i + 3] - de.w);
          }
          // which pairs of the warp's kept rows and these 32 streamed rows see one another
          bool whole = c + 32 <= s.rows;
          uint32_t see = bits(0, s.rows - c);
          const int r0 = w.row0 + (warp & 3) * 32, c0 = s.row0 + c;
          if constexpr (kKeys) {
            const int p = c0 + w.shift;
            if (!all_seen(a.mask, p, p + 31, r0)) {
              whole = false;
              see &= bits(cs.lo - p, cs.hi + 1 - p);
            }
          } else {
            const int p = r0 + w.shift;
            if (!all_seen(a.mask, p, p + 31, c0)) {
              whole = false;
              see &= seen_keys(a.mask, p + lane, c0);
            }
          }
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see >> i & 1)) x[i] = y[i] = 0.f;
          }
          uint32_t pk[16];
          if constexpr (kKeys) {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack16<T>(x[2 * i], x[2 * i + 1]);
            tmem_st16(scores + c / 2, pk);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack16<T>(y[2 * i], y[2 * i + 1]);
          tmem_st16(scores + 64 + c / 2, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ready + 8 * g);
      }
      if (!ok) break;
      if (w.count) {
        if (!(ok = mbar_wait(acc_full, nk & 1, s_abort))) break;
        tc_fence_after();
      }
      const int64_t at = (((int64_t)(kKeys ? w.e.k0 : w.e.q0) + w.row0 + row) * (kKeys ? a.kv_heads : a.heads) + w.h) * a.D;
      if (kGroups == 1 || g == 0)
        gradient_row<T, DP>(lanes + Sh::kColAcc, w.count > 0, live, a.scale, static_cast<T*>(a.d1) + at, a.D, a.sectors);
      if (kKeys && g == kGroups - 1)
        gradient_row<T, DP>(lanes + Sh::kColAcc + DP, w.count > 0, live, 1.f, static_cast<T*>(a.d2) + at, a.D, a.sectors);
      if (w.count) {
        tc_fence_before();
        mbar_arrive(acc_empty);
        ++nk;
      }
      n += w.count;
    }
  }
  const int64_t first = a.B > 0 ? a.offsets[a.B] : 0;
  const int64_t values = (int64_t)(kKeys ? a.kv_heads : a.heads) * a.D;
  zero_rows(a.d1, first, kKeys ? a.n_kv : a.n_q, values);
  if (kKeys) zero_rows(a.d2, first, a.n_kv, values);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, Sh::kColumns);
  }
  if (threadIdx.x == 0 && *s_abort) record_error(a.hdr, kDevWaitTimeout);
}

struct BwdWorkspace {
  WsHeader* hdr;
  TileItem *queries, *keys;
  float* delta;
  size_t bytes;
};
BwdWorkspace carve_backward(void* base, int64_t n_q, int64_t n_kv, int B, int heads) {
  BwdWorkspace w;
  char* p = static_cast<char*>(base);
  size_t off = 256;
  const auto take = [&](size_t bytes) {
    char* at = p + off;
    off = (off + bytes + 255) & ~(size_t)255;
    return at;
  };
  w.hdr = reinterpret_cast<WsHeader*>(p);
  w.queries = reinterpret_cast<TileItem*>(take((max_tiles(n_q, B) + 1) * sizeof(TileItem)));
  w.keys = reinterpret_cast<TileItem*>(take((max_tiles(n_kv, B) + 1) * sizeof(TileItem)));
  w.delta = reinterpret_cast<float*>(take((size_t)n_q * heads * sizeof(float)));
  w.bytes = off;
  return w;
}

template <typename T, int DP, int kGroups, bool kKeys>
cudaError_t run(const BwdArgs& a, int64_t items, const CUtensorMap& k1, const CUtensorMap& k2, const CUtensorMap& s1,
                const CUtensorMap& s2, cudaStream_t s) {
  using Sh = BwdShape<DP, kGroups, kKeys>;
  const auto kernel = k_attn_backward<T, DP, kGroups, kKeys>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::kSmem);
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
cudaError_t run_backward(const AttnCall& c, const BwdWorkspace& ws, cudaStream_t s) {
  PlanLists lists = {};
  lists.queries = ws.queries;
  lists.keys = ws.keys;
  cudaError_t e = launch_attention_plan(c, ws.hdr, lists, s);
  if (e != cudaSuccess) return e;
  const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  // without queries (or keys) no item has a tile of the other: their maps are not used
  CUtensorMap q = {}, k = {}, v = {}, d = {};
  if (c.n_q > 0 && (!attention_map(&q, c.q, bf16, c.n_q, c.heads, c.D, c.q_token, c.q_head) ||
                    !attention_map(&d, c.dout, bf16, c.n_q, c.heads, c.D, c.do_token, c.do_head)))
    return cudaErrorInvalidValue;
  if (c.n_kv > 0 && (!attention_map(&k, c.k, bf16, c.n_kv, c.kv_heads, c.D, c.k_token, c.k_head) ||
                     !attention_map(&v, c.v, bf16, c.n_kv, c.kv_heads, c.D, c.v_token, c.v_head)))
    return cudaErrorInvalidValue;
  if (c.n_q == 0) q = k, d = v;
  if (c.n_kv == 0) k = q, v = d;
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
  a.delta = ws.delta;
  a.B = c.B;
  a.hdr = ws.hdr;
  a.sectors = ((reinterpret_cast<uintptr_t>(c.dq) | reinterpret_cast<uintptr_t>(c.dk) | reinterpret_cast<uintptr_t>(c.dv)) &
               31) == 0 && c.D % 16 == 0;
  if (c.n_q > 0) {
    a.d1 = c.dq;
    a.d2 = nullptr;
    a.offsets = c.q_offsets;
    a.items = ws.queries;
    if ((e = run<T, DP, 1, false>(a, max_tiles(c.n_q, c.B) * c.heads, q, d, k, v, s)) != cudaSuccess) return e;
  }
  if (c.n_kv > 0) {
    a.d1 = c.dk;
    a.d2 = c.dv;
    a.offsets = c.kv_offsets;
    a.items = ws.keys;
    if ((e = run<T, DP, DP == 64 ? 1 : 2, true>(a, max_tiles(c.n_kv, c.B) * c.kv_heads, k, v, q, d, s)) != cudaSuccess)
      return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t attention_backward_bytes(const AttnCall& c) {
  return carve_backward(nullptr, c.n_q, c.n_kv, c.B, c.heads).bytes;
}

cudaError_t launch_attention_backward(const AttnCall& c, void* workspace, cudaStream_t s) {
  const BwdWorkspace ws = carve_backward(workspace, c.n_q, c.n_kv, c.B, c.heads);
  if (c.dtype == FPS_DTYPE_BF16)
    return c.D <= 64 ? run_backward<__nv_bfloat16, 64>(c, ws, s) : run_backward<__nv_bfloat16, 128>(c, ws, s);
  return c.D <= 64 ? run_backward<__half, 64>(c, ws, s) : run_backward<__half, 128>(c, ws, s);
}

}  // namespace fpstok
