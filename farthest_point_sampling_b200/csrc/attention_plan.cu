// Tile lists of the packed attention: which rows of which event a work item
// takes.  The offsets live on the device, so the list is made there; its
// length is bounded by rows / 128 + events.
#include "attention_plan.h"

#include <atomic>

#include "attention_few.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"

namespace fpstok {

namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return x - v + (warp ? s_warp[warp - 1] : 0);  // exclusive
}

// Sorts the first `count` (a power of two) keys in shared memory, largest
// first (bitonic).
__device__ __forceinline__ void block_sort(uint64_t* s, int count) {
  const int i = threadIdx.x;
  for (int k = 2; k <= count; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      const int x = i ^ j;
      __syncthreads();
      if (x > i && x < count) {
        const uint64_t a = s[i], b = s[x];
        if ((a < b) == ((i & k) == 0)) {
          s[i] = b;
          s[x] = a;
        }
      }
    }
  __syncthreads();
}

// NaN in `count` rows from `first` on, by threads `thread` of `threads`.
__device__ __forceinline__ void void_rows(const PlanRows& w, int64_t n, int64_t first, int64_t count, int thread,
                                          int threads) {
  const uint32_t nan2 = 0x7fff7fffu;  // two 16-bit NaN, of either type
  for (int x = 0; x < 2; ++x) {
    if (!w.rows[x]) continue;
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(w.rows[x]) + first * w.values * 2);
    for (int64_t e = thread; e < count * w.values / 8; e += threads) p[e] = make_uint4(nan2, nan2, nan2, nan2);
  }
  if (w.lse)
    for (int h = 0; h < w.heads; ++h)
      for (int64_t e = thread; e < count; e += threads) w.lse[(int64_t)h * n + first + e] = __uint_as_float(0x7fffffffu);
}

// The rows (of `off`, n in all) of the events above max_tokens among the first
// `taken`, a warp each, and of all events from there on.  By the whole block,
// and only where there are such: a call that is wrong need not be fast.
__device__ __forceinline__ void void_events(const PlanRows& w, const int64_t* off, const int64_t* q_off, const int64_t* k_off,
                                         int taken, int B, int64_t n, int max_tokens) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < taken; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const bool above = b < taken && max_tokens > 0 &&
                       (q_off[b + 1] - q_off[b] > max_tokens || k_off[b + 1] - k_off[b] > max_tokens);
    uint32_t left = __ballot_sync(kFull, above);
    while (left) {
      const int64_t first = off[b - lane + __ffs(left) - 1], end = off[b - lane + __ffs(left)];
      void_rows(w, n, first, end - first, lane, 32);
      left &= left - 1;
    }
  }
  if (taken < B) {
    const int64_t first = taken > 0 ? off[taken] : 0;  // the end of an event that was taken
    void_rows(w, n, first, n - first, threadIdx.x, kPlanThreads);
  }
}

enum PlanList { kPlanQueries, kPlanKeys, kPlanUnits, kPlanShorts };

// One block per list.  A pass takes 1024 events, one per thread: their items
// are counted and scanned, then all threads write the pass's items, each
// finding its event by bisection in shared memory, so that one long event does
// not keep one thread.
__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const int64_t* __restrict__ q_off,
                                                            const int64_t* __restrict__ k_off, int B, int64_t n_q,
                                                            int64_t n_kv, int max_tokens, int group, AttnMask mask,
                                                            WsHeader* hdr, const PlanLists lists) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_warp[32];
  __shared__ int s_start[kPlanThreads];
  __shared__ TileItem s_event[kPlanThreads];
  __shared__ uint64_t s_sort[kPlanThreads];
  const int tid = threadIdx.x;
  // forward: queries, units; backward: queries, keys, shorts
  const int kind = blockIdx.x == 0 ? kPlanQueries : lists.units ? kPlanUnits : blockIdx.x == 1 ? kPlanKeys : kPlanShorts;
  TileItem* items = kind == kPlanQueries ? lists.queries
                    : kind == kPlanKeys  ? lists.keys
                    : kind == kPlanUnits ? lists.units
                                         : lists.shorts;
  int base = 0, slots = 0, joins = 0, error = 0, taken = B;
  if (tid == 0 && B > 0 && (q_off[0] != 0 || k_off[0] != 0)) error = kDevBadOffsets;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0, parts = 0;
    TileItem e = {};
    if (b < B) {
      const int64_t q0 = q_off[b], q1 = q_off[b + 1], k0 = k_off[b], k1 = k_off[b + 1];
      if (q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > n_q || k1 > n_kv) {
        error = kDevBadOffsets;
      } else if (max_tokens > 0 && (q1 - q0 > max_tokens || k1 - k0 > max_tokens)) {
        error = error ? error : kDevTooLarge;
      } else {
        e.q0 = (int)q0;
        e.nq = (int)(q1 - q0);
        e.k0 = (int)k0;
        e.nk = (int)(k1 - k0);
        if (lists.range && kind == kPlanQueries && e.nq > 0) lists.range[e.q0] = lists.range[n_q + e.q0] = 0.f;
        const bool few = lists.units && (int64_t)e.nq * group <= kFewRows;
        const bool brief = lists.shorts && e.nq <= kTile && e.nk <= kTile;
        if (kind == kPlanQueries) {
          n = few || brief ? 0 : (e.nq + kTile - 1) / kTile;
        } else if (kind == kPlanKeys) {
          n = brief ? 0 : (e.nk + kTile - 1) / kTile;
        } else if (kind == kPlanShorts) {
          n = brief;
        } else if (few && e.nq > 0) {
          n = max((few_span(mask, e.nq, e.nk).count() + lists.chunk - 1) / lists.chunk, 1);
          parts = n > 1 ? n : 0;
        }
      }
    }
    // A pass with bad offsets makes no items and ends the list: up to there
    // offsets rise, which is what bounds the items of a list by its buffer.
    if (__syncthreads_or(error == kDevBadOffsets)) {
      taken = b0;
      break;
    }
    // Long events first, so that the blocks that claim items in turn end
    // together; where no event has more than four tiles order matters little.
    if (kind <= kPlanKeys && __syncthreads_or(n > 4)) {
      s_event[tid] = e;
      s_sort[tid] = ((uint64_t)n << 32) | (uint32_t)(kPlanThreads - 1 - tid);
      int count = 2;
      while (count < min(B - b0, kPlanThreads)) count <<= 1;
      block_sort(s_sort, count);
      n = (int)(s_sort[tid] >> 32);
      e = s_event[kPlanThreads - 1 - (uint32_t)s_sort[tid]];
      __syncthreads();
    }
    if (kind == kPlanKeys && lists.slots > 0) {
      // tiles that hold a sink, or all without a window, are seen by every query
      int cuts = 1, whole = 0;
      if (n > 0) {
        whole = mask.left < kFar ? min((mask.sinks + kTile - 1) / kTile, n) : n;
        cuts = ((e.nq / lists.stream + 2) * group + lists.piece - 1) / lists.piece;
      }
      int total_parts;
      const int want = cuts > 1 ? (int)min((int64_t)whole * cuts, (int64_t)lists.slots + 1) : 0;
      const int slot = slots + block_scan(want, s_warp, &total_parts);
      if (cuts > 1 && slot + want > lists.slots) {  // no room, which the host's count rules out
        cuts = 1;
        for (int i = slot; i < lists.slots; ++i) lists.key_joins[i] = JoinItem{0, 0, 0, 0};
      }
      e.pad[0] = cuts;
      e.pad[1] = whole;
      e.pad[2] = slot;
      if (cuts > 1) n += whole * (cuts - 1);
      slots = min(slots + total_parts, lists.slots);
    }
    int total;
    s_start[tid] = block_scan(n, s_warp, &total);
    if (kind == kPlanUnits) {
      int total_parts, total_joins;
      const int slot = slots + block_scan(parts, s_warp, &total_parts);
      const int join = joins + block_scan(parts > 0, s_warp, &total_joins);
      e.pad[0] = n;
      e.pad[1] = slot;
      if (parts) lists.joins[join] = JoinItem{e.q0, e.nq, slot, parts};
      slots += total_parts;
      joins += total_joins;
    }
    s_event[tid] = e;
    __syncthreads();
    for (int i = tid; i < total; i += kPlanThreads) {
      int lo = 0, hi = kPlanThreads - 1;  // the last event of the pass that starts at or before i
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s_start[m] <= i) lo = m; else hi = m - 1;
      }
      TileItem it = s_event[lo];
      it.t = i - s_start[lo];
      // causal: the last queries of an event see most
      if (kind == kPlanKeys) {
        const int cuts = lists.slots > 0 ? it.pad[0] : 1, whole = it.pad[1], slot = it.pad[2], at = it.t;
        it.pad[0] = 0;
        it.pad[1] = -1;
        it.pad[2] = -1;
        if (cuts > 1 && at < whole * cuts) {
          it.t = at / cuts;
          const int piece = at - it.t * cuts, rows = min(kTile, it.nk - it.t * kTile);
          int lo, hi;
          queries_of(mask, it.t * kTile, rows, it.nk - it.nq, it.nq, &lo, &hi);
          const int all = hi > lo ? (hi - (lo & ~15) + lists.stream - 1) / lists.stream * group : 0;
          const int each = all > 0 ? (all + cuts - 1) / cuts : 1, pieces = max((all + each - 1) / each, 1);
          JoinItem j = {0, 0, 0, 0};
          if (pieces > 1 && piece < pieces) {
            it.pad[0] = piece * each;
            it.pad[1] = min(it.pad[0] + each, all);
            it.pad[2] = slot + at;
            if (piece == 0) j = JoinItem{it.k0 + it.t * kTile, rows, slot + at, pieces};
          } else if (piece > 0) {
            it.pad[2] = -2;
          }
          lists.key_joins[slot + at] = j;
        } else if (cuts > 1) {
          it.t = whole + at - whole * cuts;
        }
      }
      if (kind == kPlanQueries && mask.causal) it.t = (it.nq + kTile - 1) / kTile - 1 - it.t;
      items[base + i] = it;
    }
    base += total;
    __syncthreads();
  }
  error = __syncthreads_or(error == kDevBadOffsets) ? kDevBadOffsets : __syncthreads_or(error) ? kDevTooLarge : 0;
  if (error && kind == kPlanQueries) void_events(lists.of_queries, q_off, q_off, k_off, taken, B, n_q, max_tokens);
  if (error && kind == kPlanKeys) void_events(lists.of_keys, k_off, q_off, k_off, taken, B, n_kv, max_tokens);
  if (tid == 0) {
    const int list = kind == kPlanQueries ? kQueryTiles
                     : kind == kPlanKeys  ? kKeyTiles
                     : kind == kPlanUnits ? kFewUnits
                                          : kShortEvents;
    hdr->next_item[list] = 0;
    hdr->n_items[list] = base;
    if (kind == kPlanUnits) hdr->n_items[kFewJoins] = joins;
    if (kind == kPlanKeys) hdr->n_items[kKeySlots] = slots;
    if (kind == kPlanQueries) {  // every block sees the same errors; one writes the status word
      hdr->status = error;
      hdr->detail = 0;
    }
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

}  // namespace

cudaError_t allow_shared_memory(const void* kernel, int bytes) {
  // a few kernels, each found after as many compares; a lost race sets one twice
  struct Entry {
    std::atomic<const void*> kernel;
    std::atomic<uint64_t> devices;  // bit per device
  };
  static Entry entries[64];
  int device;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  Entry* at = nullptr;
  for (Entry& x : entries) {
    const void* free_slot = nullptr;
    if (x.kernel.load(std::memory_order_acquire) == kernel ||
        (x.kernel.compare_exchange_strong(free_slot, kernel) || free_slot == kernel)) {
      at = &x;
      break;
    }
  }
  if (at && device < 64 && (at->devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && at) at->devices.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_attention_plan(const AttnCall& c, WsHeader* hdr, const PlanLists& lists, cudaStream_t s) {
  count_launch();
  k_attn_plan<<<lists.shorts ? 3 : lists.units ? 2 : 1, kPlanThreads, 0, s>>>(
      c.q_offsets, c.kv_offsets, c.B, c.n_q, c.n_kv, c.max_tokens, c.group, c.mask, hdr, lists);
  return cudaGetLastError();
}

bool attention_map(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int heads, int D, int64_t token_stride,
                   int64_t head_stride) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, 1, 64};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fpstok
