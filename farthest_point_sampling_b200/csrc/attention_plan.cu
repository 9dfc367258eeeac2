// Tile lists of the packed attention: which rows of which event a work item
// takes.  The offsets live on the device, so the list is made there; its
// length is bounded by rows / 128 + events.
#include "attention_plan.h"

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

// Block 0 makes the query list, block 1 the key list.  A pass takes 1024
// events, one per thread: their tiles are counted and scanned, then all
// threads write the pass's items, each finding its event by bisection in
// shared memory, so that one long event does not keep one thread.
__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const int64_t* __restrict__ q_off,
                                                            const int64_t* __restrict__ k_off, int B, int64_t n_q,
                                                            int64_t n_kv, int max_tokens, WsHeader* hdr,
                                                            TileItem* queries, TileItem* keys) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_warp[32];
  __shared__ int s_start[kPlanThreads + 1];
  __shared__ TileItem s_event[kPlanThreads];
  const int tid = threadIdx.x;
  const bool key_list = blockIdx.x == 1;
  TileItem* items = key_list ? keys : queries;
  int base = 0, error = 0;
  if (tid == 0 && B > 0 && (q_off[0] != 0 || k_off[0] != 0)) error = kDevBadOffsets;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int tiles = 0;
    if (b < B) {
      const int64_t q0 = q_off[b], q1 = q_off[b + 1], k0 = k_off[b], k1 = k_off[b + 1];
      if (q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > n_q || k1 > n_kv) {
        error = kDevBadOffsets;
      } else if (max_tokens > 0 && (q1 - q0 > max_tokens || k1 - k0 > max_tokens)) {
        error = error ? error : kDevTooLarge;
      } else {
        s_event[tid] = TileItem{(int)q0, (int)(q1 - q0), (int)k0, (int)(k1 - k0), 0, {0, 0, 0}};
        tiles = (int)(((key_list ? k1 - k0 : q1 - q0) + kTile - 1) / kTile);
      }
    }
    // A pass with bad offsets makes no items and ends the list: up to there
    // offsets rise, which is what bounds the items of a list by max_tiles().
    if (__syncthreads_or(error == kDevBadOffsets)) break;
    int total;
    s_start[tid] = block_scan(tiles, s_warp, &total);
    __syncthreads();
    for (int e = tid; e < total; e += kPlanThreads) {
      int lo = 0, hi = kPlanThreads - 1;  // the last event of the pass that starts at or before e
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s_start[m] <= e) lo = m; else hi = m - 1;
      }
      TileItem it = s_event[lo];
      it.t = e - s_start[lo];
      items[base + e] = it;
    }
    base += total;
    __syncthreads();
  }
  // one writer of the status word per block, the query block's after its reset
  error = __syncthreads_or(error == kDevBadOffsets) ? kDevBadOffsets : __syncthreads_or(error) ? kDevTooLarge : 0;
  if (tid == 0) {
    hdr->n_items[key_list ? kKeyTiles : kQueryTiles] = base;
    if (!key_list) {
      hdr->status = error;
      hdr->detail = 0;
      hdr->next_item[0] = 0;
      hdr->next_item[1] = 0;
      hdr->next_item[2] = 0;
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

cudaError_t launch_attention_plan(const AttnCall& c, WsHeader* hdr, TileItem* queries, TileItem* keys,
                                  cudaStream_t s) {
  count_launch();
  k_attn_plan<<<keys ? 2 : 1, kPlanThreads, 0, s>>>(c.q_offsets, c.kv_offsets, c.B, c.n_q, c.n_kv, c.max_tokens, hdr,
                                                    queries, keys);
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
