// Attention of packed events, forward, on the tensor cores.
//
// One work item is a tile of 128 queries of one event and one head.  With S =
// Q K^T over a tile of 128 keys, the running maximum m and sum l of the
// softmax give
//   P = exp2(c S - c m),  l <- l f + sum P,  O <- O f + P V,  f = exp2(c (m_old - m)),
// c = scale log2(e), and the output is O / l, lse = m scale + ln l.
//
// A block is six warps: one thread loads Q, K and V tiles with TMA, one issues
// the tcgen05 products, and four warps do the softmax with one query row per
// thread (a TMEM lane), so no row crosses threads.  S goes to TMEM, P comes
// back over it as 16-bit operand A of the second product, O stays in TMEM
// until the item ends.  Two blocks share an SM: while one's softmax runs, the
// other's products do.  Blocks are persistent; the loader runs ahead into the
// next items.
//
// Rounding: P is rounded to the input type for P V; l sums the unrounded
// values.  O is rescaled only when m grows by more than 8 / log2 units, which
// leaves P at most 2^8: exact in the float32 accumulator and far from the
// range limits of both types.
#include <type_traits>

#include "attention_plan.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace fpstok {

namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kFwdThreads = 256;  // the softmax warp group, and one of a loading and an issuing warp (two idle)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 48;  // a thread's share after the split; launched with 128 each
constexpr int kPanel = kTile * 128;  // bytes of a 128-row panel of 64 values
constexpr uint32_t kTmemColumns = 256;
constexpr uint32_t kColO = 128;  // S (and P over it) in columns 0 .. 127

template <int DP>
struct FwdShape {
  static constexpr int kPanels = DP / 64;
  static constexpr int kStages = DP == 64 ? 2 : 1;  // of Q, K and V each: 96 KB either way, two blocks per SM
  static constexpr uint32_t kTileBytes = kPanels * kPanel;
  static constexpr size_t kSmem = 1024 + 3 * kStages * kTileBytes + 256;
};

struct FwdArgs {
  int64_t n_q;
  int heads, group, D;
  AttnMask mask;
  float scale, scale_log2;
  void* out;
  float* lse;
  const int64_t* q_offsets;
  int B, zero_tail;
  const TileItem* items;
  WsHeader* hdr;
};

// What every role of the block computes alike for one item.
struct FwdItem {
  TileItem e;
  int h, row0, rows, p0;  // head; first query of the tile in its event, queries of the tile, position of the first
  KeyTiles<kTile> keys;
};
__device__ __forceinline__ FwdItem fwd_item(const FwdArgs& a, int h, const TileItem& e) {
  FwdItem w;
  w.h = h;
  w.e = e;
  w.row0 = w.e.t * kTile;
  w.rows = min(kTile, w.e.nq - w.row0);
  w.p0 = w.row0 + w.e.nk - w.e.nq;
  w.keys = key_tiles<kTile>(a.mask, w.p0, w.p0 + w.rows - 1, w.e.nk);
  return w;
}

// Bits lo .. hi - 1 of a word, bounds clipped to 0 .. 32.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
}

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
  uint64_t* s_bar = reinterpret_cast<uint64_t*>(s_v + Sh::kStages * Sh::kTileBytes);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_bar + 16);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t q_full = bars, k_full = bars + 16, k_empty = bars + 32, v_full = bars + 48, v_empty = bars + 64,
                 s_full = bars + 80, o_full = bars + 88, drain = bars + 96, p_ready = bars + 104, q_empty = bars + 112;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 13; ++i) mbar_init(bars + 8 * i, 1);
    mbar_init(p_ready, 32 * kSoftmaxWarps);
    mbar_init(q_empty, 32 * kSoftmaxWarps);
    mbar_init(q_empty + 8, 32 * kSoftmaxWarps);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == kSoftmaxWarps + 1) tmem_alloc(smem_u32(s_tmem), kTmemColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // every role walks the block's items, and reads the next one's entry while it works on one
  ItemWalk walk(a.heads, a.hdr->n_items[kQueryTiles]);
  TileItem next = a.items[walk.more() ? walk.tile : 0];

  if (warp >= kSoftmaxWarps) {
    regs_down<kOtherRegs>();
    if (warp == kSoftmaxWarps && lane == 0) {
      // ------------------------------------------------ loads
      int n = 0, nq = 0;  // key tiles and query tiles loaded so far
      bool ok = true;
      while (walk.more() && ok) {
        const FwdItem w = fwd_item(a, walk.h, next);
        walk.advance();
        if (walk.more()) next = a.items[walk.tile];
        if (w.keys.count == 0) continue;
        const int qs = nq % Sh::kStages;
        if (nq >= Sh::kStages && !(ok = mbar_wait(q_empty + 8 * qs, ((nq / Sh::kStages) - 1) & 1, s_abort))) break;
        const int q_boxes = (w.rows + 63) / 64;
        mbar_expect(q_full + 8 * qs, q_boxes * 8192 * Sh::kPanels);
#pragma unroll 1
        for (int p = 0; p < Sh::kPanels; ++p)
#pragma unroll 1
          for (int i = 0; i < q_boxes; ++i)
            tma_load(smem_u32(s_q) + qs * Sh::kTileBytes + p * kPanel + i * 8192, &map_q, q_full + 8 * qs, p * 64, w.h,
                     w.e.q0 + w.row0 + i * 64);
        ++nq;
        const int g = w.h / a.group;
        for (int j = 0; j < w.keys.count; ++j, ++n) {
          const int st = n % Sh::kStages;
          const uint32_t round = ((n / Sh::kStages) - 1) & 1;
          const int boxes = (w.keys.extent(j) + 63) / 64;
          const int krow = w.e.k0 + w.keys.start(j);
          if (n >= Sh::kStages && !(ok = mbar_wait(k_empty + 8 * st, round, s_abort))) break;
          mbar_expect(k_full + 8 * st, boxes * 8192 * Sh::kPanels);
#pragma unroll 1
          for (int p = 0; p < Sh::kPanels; ++p)
#pragma unroll 1
            for (int i = 0; i < boxes; ++i)
              tma_load(smem_u32(s_k) + st * Sh::kTileBytes + p * kPanel + i * 8192, &map_k, k_full + 8 * st, p * 64, g,
                       krow + i * 64);
          if (n >= Sh::kStages && !(ok = mbar_wait(v_empty + 8 * st, round, s_abort))) break;
          mbar_expect(v_full + 8 * st, boxes * 8192 * Sh::kPanels);
#pragma unroll 1
          for (int p = 0; p < Sh::kPanels; ++p)
#pragma unroll 1
            for (int i = 0; i < boxes; ++i)
              tma_load(smem_u32(s_v) + st * Sh::kTileBytes + p * kPanel + i * 8192, &map_v, v_full + 8 * st, p * 64, g,
                       krow + i * 64);
        }
      }
      // after a wait that gave up: this thread's copies still in flight land first
      if (*s_abort) {
        volatile int none = 0;
        for (int i = 0; i < Sh::kStages; ++i) {
          const int lq = nq - 1 - i, lk = n - i;  // tile n may have its keys loading, not its values
          if (lq >= 0) mbar_wait(q_full + 8 * (lq % Sh::kStages), (lq / Sh::kStages) & 1, &none);
          if (lk >= 0) mbar_wait(k_full + 8 * (lk % Sh::kStages), (lk / Sh::kStages) & 1, &none);
          if (lk >= 1) mbar_wait(v_full + 8 * ((lk - 1) % Sh::kStages), ((lk - 1) / Sh::kStages) & 1, &none);
        }
      }
    } else if (warp == kSoftmaxWarps + 1 && lane == 0) {
      // ------------------------------------------------ products
      int n = 0, nq = 0;
      const int d_steps = (a.D + 15) / 16;
      const uint32_t pv_desc = mma_desc(kBf16, false, true, d_steps * 16);
      bool ok = true;
      while (walk.more() && ok) {
        const FwdItem w = fwd_item(a, walk.h, next);
        walk.advance();
        if (walk.more()) next = a.items[walk.tile];
        if (w.keys.count == 0) continue;
        const int qs = nq % Sh::kStages;
        const uint32_t q = smem_desc(smem_u32(s_q) + qs * Sh::kTileBytes, kPanel);
        if (!(ok = mbar_wait(q_full + 8 * qs, (nq / Sh::kStages) & 1, s_abort))) break;
        for (int j = 0; j <= w.keys.count; ++j) {
          if (j > 0) {  // O += P V of tile j - 1
            const int m = n + j - 1, st = m % Sh::kStages;
            const int steps = (w.keys.extent(j - 1) + 15) / 16;
            if (!(ok = mbar_wait(v_full + 8 * st, (m / Sh::kStages) & 1, s_abort))) break;
            if (!(ok = mbar_wait(p_ready, m & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t v = smem_desc(smem_u32(s_v) + st * Sh::kTileBytes, kPanel);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              if (ks < steps) mma_ts(tmem + kColO, tmem + ks * 8, v + ks * 128, pv_desc, ks > 0 || j > 1);
            mma_commit(v_empty + 8 * st);
            if (j == w.keys.count) mma_commit(o_full);
          }
          if (j < w.keys.count) {  // S = Q K^T of tile j; over P, which the product before has read
            const int m = n + j, st = m % Sh::kStages;
            const int cols = (w.keys.extent(j) + 15) / 16 * 16;
            if (!(ok = mbar_wait(k_full + 8 * st, (m / Sh::kStages) & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t k = smem_desc(smem_u32(s_k) + st * Sh::kTileBytes, kPanel);
            const uint32_t qk_desc = mma_desc(kBf16, false, false, cols);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
              const uint32_t at = ((ks >> 2) * kPanel + (ks & 3) * 32) >> 4;
              if (ks < d_steps) mma_ss(tmem, q + at, k + at, qk_desc, ks > 0);
            }
            mma_commit(k_empty + 8 * st);
            mma_commit(s_full);
          }
        }
        if (!ok) break;
        n += w.keys.count;
        ++nq;
      }
      if (*s_abort) {  // products in flight end before TMEM is freed
        volatile int none = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &none);
      }
    }
  } else {
    // ------------------------------------------------ softmax
    regs_up<kSoftmaxRegs>();
    int n = 0, nq = 0;  // key tiles and query tiles so far
    const int row = threadIdx.x;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    while (walk.more() && ok) {
      const FwdItem w = fwd_item(a, walk.h, next);
      walk.advance();
      if (walk.more()) next = a.items[walk.tile];
      const int64_t qrow = (int64_t)w.e.q0 + w.row0 + row;
      T* out = static_cast<T*>(a.out) + ((int64_t)(w.e.q0 + w.row0 + warp * 32) * a.heads + w.h) * a.D;
      const int warp_rows = min(32, w.rows - warp * 32);
      if (w.keys.count == 0) {  // nothing to see
        for (int r = lane; r < warp_rows; r += 32) {
          for (int c = 0; c < a.D; c += 8)
            *reinterpret_cast<uint4*>(out + (int64_t)r * a.heads * a.D + c) = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[(int64_t)w.h * a.n_q + qrow] = -INFINITY;
        }
        continue;
      }
      const RowSpan span = row_span(a.mask, w.p0 + row, w.e.nk);
      // keys that some row of this warp sees
      const RowSpan warp_lo = row_span(a.mask, w.p0 + warp * 32, w.e.nk);
      const RowSpan warp_hi = row_span(a.mask, w.p0 + min(warp * 32 + 31, w.rows - 1), w.e.nk);
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < w.keys.count; ++j, ++n) {
        const int st = n % Sh::kStages;
        const int k0 = w.keys.start(j), extent = w.keys.extent(j);
        const int odd = extent & 15;
        if (odd) {
          // Keys past the tile's last inside the product's step of 16: their
          // weights are 0, and their values must be finite for 0 to stay 0.
          if (!(ok = mbar_wait(v_full + 8 * st, (n / Sh::kStages) & 1, s_abort))) break;
          uint8_t* v_tile = s_v + st * Sh::kTileBytes;
          for (int e = threadIdx.x; e < (16 - odd) * 8 * Sh::kPanels; e += 32 * kSoftmaxWarps) {
            const int r = extent + e / (8 * Sh::kPanels), c = e % (8 * Sh::kPanels);
            *reinterpret_cast<uint4*>(v_tile + (c >> 3) * kPanel + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        // 32-column chunks of the tile that some row of the warp sees
        int act = 0;
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c) {
          const int first = k0 + 32 * c, last = k0 + min(32 * c + 31, extent - 1);
          if (32 * c < extent && warp_rows > 0 &&
              ((last >= warp_lo.lo && first < warp_hi.hi) || first < warp_hi.s))
            act |= 1 << c;
        }
        const bool masked = (extent & 31) != 0 || tile_masked(a.mask, w.p0, w.p0 + w.rows - 1, k0, k0 + extent);
        if (!(ok = mbar_wait(s_full, n & 1, s_abort))) break;
        tc_fence_after();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c)
          if (act >> c & 1) tmem_ld32(lanes + 32 * c, reinterpret_cast<uint32_t*>(s + 32 * c));
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c) tmem_wait_ld32(reinterpret_cast<uint32_t*>(s + 32 * c));
        if (masked) {
          const int from = span.lo - k0, width = min(span.hi - k0, extent) - from, sink = min(span.s - k0, extent);
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c)
            if (act >> c & 1) {
              const uint32_t see = bits(from - 32 * c, from + width - 32 * c) | bits(0, sink - 32 * c);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(see >> i & 1)) s[32 * c + i] = -INFINITY;
            }
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c)
          if (act >> c & 1) {
#pragma unroll
            for (int i = 32 * c; i < 32 * c + 32; i += 4) {
              m0 = max3f(m0, s[i], s[i + 1]);
              m1 = max3f(m1, s[i + 2], s[i + 3]);
            }
          }
        const float top = fmaxf(m0, m1);
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
            for (int c = 0; c < DP; c += 16) {
              uint32_t o[16];
              tmem_ld16(lanes + kColO + c, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(lanes + kColO + c, o);
            }
          }
        }
        const float base = m_used == -INFINITY ? 0.f : m_used * a.scale_log2;
        const float2 base2 = make_float2(-base, -base);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c) {
          uint32_t pk[16];
          if (act >> c & 1) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float2 e = fma2(make_float2(s[32 * c + i], s[32 * c + i + 1]), scale2, base2);
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              sum = add2(sum, e);
              pk[i / 2] = pack16<T>(e.x, e.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0;
          }
          if (32 * c < extent) tmem_st16(lanes + 16 * c, pk);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
      }
      if (!ok) break;
      const int qs = nq % Sh::kStages;
      if (!(ok = mbar_wait(o_full, nq & 1, s_abort))) break;
      ++nq;
      tc_fence_after();
      // O / l to the item's query tile in shared memory, which no product
      // reads any more, then to memory with whole rows per instruction; a
      // warp only touches its own rows.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint8_t* stage = s_q + qs * Sh::kTileBytes;
#pragma unroll
      for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        tmem_ld32(lanes + kColO + c, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint4 v;
          uint32_t* pv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            pv[q] = l == 0.f ? 0u
                             : pack16<T>(__uint_as_float(o[i + 2 * q]) * inv, __uint_as_float(o[i + 2 * q + 1]) * inv);
          const int k = (c + i) / 8;
          *reinterpret_cast<uint4*>(stage + (k >> 3) * kPanel + row * 128 + (((k & 7) ^ (row & 7)) << 4)) = v;
        }
      }
      tc_fence_before();
      __syncwarp();
      constexpr int kChunks = DP / 8, kRowsAtOnce = 32 / kChunks;
      const int chunk = lane % kChunks, first = lane / kChunks;
      uint4 v[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int rr = warp * 32 + first + i * kRowsAtOnce;
        v[i] = *reinterpret_cast<const uint4*>(stage + (chunk >> 3) * kPanel + rr * 128 +
                                               (((chunk & 7) ^ (rr & 7)) << 4));
      }
      fence_async_smem();  // these reads and writes before the next tile's load
      mbar_arrive(q_empty + 8 * qs);
      if (chunk * 8 < a.D) {
        const int64_t row_values = (int64_t)a.heads * a.D;
        T* to = out + first * row_values + chunk * 8;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          if (first + i * kRowsAtOnce < warp_rows) *reinterpret_cast<uint4*>(to + i * kRowsAtOnce * row_values) = v[i];
      }
      if (lane < warp_rows && a.lse)
        a.lse[(int64_t)w.h * a.n_q + qrow] = l == 0.f ? -INFINITY : fmaf(m_used, a.scale, logf(l));
    }
  }
  if (a.zero_tail) zero_rows(a.out, a.B > 0 ? a.q_offsets[a.B] : 0, a.n_q, (int64_t)a.heads * a.D);
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, kTmemColumns);
  }
  if (threadIdx.x == 0 && *s_abort) record_error(a.hdr, kDevWaitTimeout);
}

struct FwdWorkspace {
  WsHeader* hdr;
  TileItem* items;
  size_t bytes;
};
FwdWorkspace carve_forward(void* base, int64_t n_q, int B) {
  FwdWorkspace w;
  char* p = static_cast<char*>(base);
  w.hdr = reinterpret_cast<WsHeader*>(p);
  w.items = reinterpret_cast<TileItem*>(p + 256);
  w.bytes = 256 + (size_t)(max_tiles(n_q, B) + 1) * sizeof(TileItem);
  w.bytes = (w.bytes + 255) & ~(size_t)255;
  return w;
}

template <typename T, int DP>
cudaError_t run_forward(const AttnCall& c, const FwdWorkspace& ws, cudaStream_t s) {
  cudaError_t e = launch_attention_plan(c, ws.hdr, ws.items, nullptr, s);
  if (e != cudaSuccess || c.n_q == 0) return e;
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
  a.zero_tail = c.zero_tail;
  a.items = ws.items;
  a.hdr = ws.hdr;
  const auto kernel = k_attn_forward<T, DP>;
  constexpr int smem = (int)FwdShape<DP>::kSmem;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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

}  // namespace

size_t attention_forward_bytes(int64_t n_q, int B) { return carve_forward(nullptr, n_q, B).bytes; }

cudaError_t launch_attention_forward(const AttnCall& c, void* workspace, cudaStream_t s) {
  const FwdWorkspace ws = carve_forward(workspace, c.n_q, c.B);
  if (c.dtype == FPS_DTYPE_BF16)
    return c.D <= 64 ? run_forward<__nv_bfloat16, 64>(c, ws, s) : run_forward<__nv_bfloat16, 128>(c, ws, s);
  return c.D <= 64 ? run_forward<__half, 64>(c, ws, s) : run_forward<__half, 128>(c, ws, s);
}

}  // namespace fpstok
