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
constexpr int kFwdThreads = 32 * (kSoftmaxWarps + 2);
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
  KeyTiles keys;
};
__device__ __forceinline__ FwdItem fwd_item(const FwdArgs& a, int item) {
  FwdItem w;
  const int tile = item / a.heads;
  w.h = item - tile * a.heads;
  w.e = a.items[tile];
  w.row0 = w.e.t * kTile;
  w.rows = min(kTile, w.e.nq - w.row0);
  w.p0 = w.row0 + w.e.nk - w.e.nq;
  w.keys = key_tiles<kTile>(a.mask, w.p0, w.p0 + w.rows - 1, w.e.nk);
  return w;
}

// Scores of 32 columns from column c0 of the tile on: those outside [from,
// from + width) and not below sink to -inf.
__device__ __forceinline__ void hide(float* s, int c0, int from, int width, int sink) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int c = c0 + i;
    if (!((c >= from && c - from < width) || c < sink)) s[i] = -INFINITY;
  }
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
  const uint32_t q_full = bars, q_empty = bars + 16, k_full = bars + 32, k_empty = bars + 48, v_full = bars + 64,
                 v_empty = bars + 80, s_full = bars + 96, p_ready = bars + 104, o_full = bars + 112;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 12; ++i) mbar_init(bars + 8 * i, 1);
    mbar_init(s_full, 1);
    mbar_init(p_ready, 32 * kSoftmaxWarps);
    mbar_init(o_full, 1);
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
  const int n_items = a.hdr->n_items[kQueryTiles] * a.heads;

  if (warp == kSoftmaxWarps) {
    // ------------------------------------------------ loads
    if (lane == 0) {
      int n = 0, nq = 0;  // key tiles and query tiles loaded so far
      for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
        const FwdItem w = fwd_item(a, item);
        if (w.keys.count == 0) continue;
        const int qs = nq % Sh::kStages;
        if (nq >= Sh::kStages && !mbar_wait(q_empty + 8 * qs, ((nq / Sh::kStages) - 1) & 1, s_abort)) break;
        const int q_boxes = (w.rows + 63) / 64;
        mbar_expect(q_full + 8 * qs, q_boxes * 64 * 128 * Sh::kPanels);
        for (int p = 0; p < Sh::kPanels; ++p)
          for (int i = 0; i < q_boxes; ++i)
            tma_load(smem_u32(s_q) + qs * Sh::kTileBytes + p * kPanel + i * 8192, &map_q, q_full + 8 * qs, p * 64, w.h,
                     w.e.q0 + w.row0 + i * 64);
        ++nq;
        const int g = w.h / a.group;
        bool ok = true;
        for (int j = 0; j < w.keys.count && ok; ++j, ++n) {
          const int st = n % Sh::kStages;
          const uint32_t round = ((n / Sh::kStages) - 1) & 1;
          const int k0 = w.keys.tile(j) * kTile;
          const int boxes = (min(kTile, w.e.nk - k0) + 63) / 64;
          const uint32_t bytes = boxes * 64 * 128 * Sh::kPanels;
          if (n >= Sh::kStages && !(ok = mbar_wait(k_empty + 8 * st, round, s_abort))) break;
          mbar_expect(k_full + 8 * st, bytes);
          for (int p = 0; p < Sh::kPanels; ++p)
            for (int i = 0; i < boxes; ++i)
              tma_load(smem_u32(s_k) + st * Sh::kTileBytes + p * kPanel + i * 8192, &map_k, k_full + 8 * st, p * 64, g,
                       w.e.k0 + k0 + i * 64);
          if (n >= Sh::kStages && !(ok = mbar_wait(v_empty + 8 * st, round, s_abort))) break;
          mbar_expect(v_full + 8 * st, bytes);
          for (int p = 0; p < Sh::kPanels; ++p)
            for (int i = 0; i < boxes; ++i)
              tma_load(smem_u32(s_v) + st * Sh::kTileBytes + p * kPanel + i * 8192, &map_v, v_full + 8 * st, p * 64, g,
                       w.e.k0 + k0 + i * 64);
        }
        if (!ok) break;
      }
      // after a wait that gave up: this thread's copies still in flight land first
      if (*s_abort) {
        volatile int none = 0;
        for (int i = 0; i < Sh::kStages; ++i) {
          const int lq = nq - 1 - i, lk = n - 1 - i;
          if (lq >= 0) mbar_wait(q_full + 8 * (lq % Sh::kStages), (lq / Sh::kStages) & 1, &none);
          if (lk >= 0) mbar_wait(k_full + 8 * (lk % Sh::kStages), (lk / Sh::kStages) & 1, &none);
          if (lk >= 0) mbar_wait(v_full + 8 * (lk % Sh::kStages), (lk / Sh::kStages) & 1, &none);
        }
      }
    }
  } else if (warp == kSoftmaxWarps + 1) {
    // ------------------------------------------------ products
    if (lane == 0) {
      int n = 0, nq = 0;
      const int k_steps = (a.D + 15) / 16;
      const uint32_t pv_desc = mma_desc(kBf16, false, true, k_steps * 16);
      bool ok = true;
      for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
        const FwdItem w = fwd_item(a, item);
        if (w.keys.count == 0) continue;
        const int qs = nq % Sh::kStages;
        const uint32_t q_addr = smem_u32(s_q) + qs * Sh::kTileBytes;
        if (!(ok = mbar_wait(q_full + 8 * qs, (nq / Sh::kStages) & 1, s_abort))) break;
        for (int j = 0; j <= w.keys.count; ++j) {
          if (j > 0) {  // O += P V of tile j - 1
            const int m = n + j - 1, st = m % Sh::kStages;
            const int steps = (min(kTile, w.e.nk - w.keys.tile(j - 1) * kTile) + 15) / 16;
            if (!(ok = mbar_wait(v_full + 8 * st, (m / Sh::kStages) & 1, s_abort))) break;
            if (!(ok = mbar_wait(p_ready, m & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t v_addr = smem_u32(s_v) + st * Sh::kTileBytes;
            for (int ks = 0; ks < steps; ++ks)
              mma_ts(tmem + kColO, tmem + ks * 8, smem_desc(v_addr + ks * 2048, kPanel), pv_desc, j > 1 || ks > 0);
            mma_commit(v_empty + 8 * st);
            if (j == w.keys.count) mma_commit(o_full);
          }
          if (j < w.keys.count) {  // S = Q K^T of tile j; over P, which the product before has read
            const int m = n + j, st = m % Sh::kStages;
            const int cols = (min(kTile, w.e.nk - w.keys.tile(j) * kTile) + 15) / 16 * 16;
            if (!(ok = mbar_wait(k_full + 8 * st, (m / Sh::kStages) & 1, s_abort))) break;
            tc_fence_after();
            const uint32_t k_addr = smem_u32(s_k) + st * Sh::kTileBytes;
            const uint32_t qk_desc = mma_desc(kBf16, false, false, cols);
            for (int ks = 0; ks < k_steps; ++ks) {
              const uint32_t at = (ks >> 2) * kPanel + (ks & 3) * 32;
              mma_ss(tmem, smem_desc(q_addr + at, kPanel), smem_desc(k_addr + at, kPanel), qk_desc, ks > 0);
            }
            mma_commit(k_empty + 8 * st);
            mma_commit(s_full);
            if (j == w.keys.count - 1) mma_commit(q_empty + 8 * qs);
          }
        }
        if (!ok) break;
        n += w.keys.count;
        ++nq;
      }
      if (*s_abort) {  // products in flight end before TMEM is freed
        volatile int none = 0;
        mbar_init(bars + 120, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mma_commit(bars + 120);
        mbar_wait(bars + 120, 0, &none);
      }
    }
  } else {
    // ------------------------------------------------ softmax
    int n = 0, done = 0;  // key tiles and items so far
    const int row = threadIdx.x;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      const FwdItem w = fwd_item(a, item);
      const int64_t qrow = (int64_t)w.e.q0 + w.row0 + row;
      const int p = w.p0 + row;
      const RowSpan span = row_span(a.mask, p, w.e.nk);
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < w.keys.count; ++j, ++n) {
        const int st = n % Sh::kStages;
        const int k0 = w.keys.tile(j) * kTile;
        const int valid = min(kTile, w.e.nk - k0);
        const int odd = valid & 15;
        if (odd) {
          // Keys past the event's last inside the product's step of 16: their
          // weights are 0, and their values must be finite for 0 to stay 0.
          if (!(ok = mbar_wait(v_full + 8 * st, (n / Sh::kStages) & 1, s_abort))) break;
          uint8_t* v_tile = s_v + st * Sh::kTileBytes;
          for (int e = threadIdx.x; e < (16 - odd) * 8 * Sh::kPanels; e += 32 * kSoftmaxWarps) {
            const int r = valid + e / (8 * Sh::kPanels), c = e % (8 * Sh::kPanels);
            *reinterpret_cast<uint4*>(v_tile + (c >> 3) * kPanel + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        if (!(ok = mbar_wait(s_full, n & 1, s_abort))) break;
        tc_fence_after();
        // S is read from TMEM twice, 32 columns at a time with the next 32 on
        // their way: once for the row's maximum, once for the weights.
        const bool masked = valid < kTile || tile_masked(a.mask, w.p0, w.p0 + w.rows - 1, k0, k0 + valid);
        const int from = span.lo - k0, width = min(span.hi - k0, valid) - from, sink = min(span.s - k0, valid);
        const int chunks = (valid + 31) >> 5;
        float s[2][32];
        tmem_ld32(lanes, reinterpret_cast<uint32_t*>(s[0]));
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c)
          if (c < chunks) {
            tmem_wait_ld32(reinterpret_cast<uint32_t*>(s[c & 1]));
            if (c + 1 < kTile / 32 && c + 1 < chunks)
              tmem_ld32(lanes + 32 * (c + 1), reinterpret_cast<uint32_t*>(s[(c + 1) & 1]));
            float* v = s[c & 1];
            if (masked) hide(v, 32 * c, from, width, sink);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              m0 = max3f(m0, v[i], v[i + 1]);
              m1 = max3f(m1, v[i + 2], v[i + 3]);
            }
          }
        tmem_ld32(lanes, reinterpret_cast<uint32_t*>(s[0]));
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
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < kTile / 32; ++c)
          if (c < chunks) {
            tmem_wait_ld32(reinterpret_cast<uint32_t*>(s[c & 1]));
            if (c + 1 < kTile / 32 && c + 1 < chunks)
              tmem_ld32(lanes + 32 * (c + 1), reinterpret_cast<uint32_t*>(s[(c + 1) & 1]));
            float* v = s[c & 1];
            if (masked) hide(v, 32 * c, from, width, sink);
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float e0 = exp2_approx(fmaf(v[i], a.scale_log2, -base));
              const float e1 = exp2_approx(fmaf(v[i + 1], a.scale_log2, -base));
              l0 += e0;
              l1 += e1;
              pk[i / 2] = pack16<T>(e0, e1);
            }
            tmem_st16(lanes + 16 * c, pk);  // columns whose S this pass has read already
          }
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_ready);
      }
      if (!ok) break;
      const bool live = row < w.rows;
      T* out = static_cast<T*>(a.out) + (qrow * a.heads + w.h) * a.D;
      if (w.keys.count) {
        if (!(ok = mbar_wait(o_full, done & 1, s_abort))) break;
        ++done;
        tc_fence_after();
      }
      const float inv = w.keys.count == 0 || l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        if (w.keys.count) {
          tmem_ld32(lanes + kColO + c, o);
          tmem_wait_ld32(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            if (c + i < a.D) {
              uint4 v;
              uint32_t* pv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                pv[q] = pack16<T>(l == 0.f ? 0.f : __uint_as_float(o[i + 2 * q]) * inv,
                                  l == 0.f ? 0.f : __uint_as_float(o[i + 2 * q + 1]) * inv);
              *reinterpret_cast<uint4*>(out + c + i) = v;
            }
        }
      }
      tc_fence_before();
      if (live && a.lse) a.lse[(int64_t)w.h * a.n_q + qrow] = l == 0.f ? -INFINITY : fmaf(m_used, a.scale, logf(l));
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
