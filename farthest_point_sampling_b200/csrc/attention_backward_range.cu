// Attention of packed events, backward in float16: how large an event's score
// gradients can be.
//
// P_ij is about 1 / n with n keys in sight, and dS_ij = P_ij (dP_ij - D_i) that
// times |dO|.  Rounded to float16 for their products as they are, they leave
// its normal range (from 6e-5 up) for long events or small gradients: 12000
// keys and |dO| of 0.001 left dQ 14 times the error of rounding it once, 200000
// and 0.01 43 times (now 1.0 and 1.3).  So the products take
//   P' = 2^14 P   and   dS' = P' c (dP - D),
// and the sums are scaled back in float32 where they are stored.  With
// M = max_i |dO_i| max_j |V_j| over an event, |dP_ij| <= M and |D_i| <= M, so for
// a power of two c <= 1 / M nothing passes 2^15 < 65504.  What is far below M
// stays exact to 2^-25 of it.  bfloat16 has the range of float32, and its
// products take P and dS as they are.
//
// This kernel forms both maxima of every event, a block for each head of a tile
// in the lists of the call.  Bound by memory: it reads dO and V once more than
// the gradients need.  2048 events of up to 128 tokens, 12 heads of 64: 133 us,
// 5.2 TB/s, beside 725 (the maxima of a unit's tiles taken in its own kernel made
// that 857); 64 track events of up to 20000 tokens, 8 query and 2 key heads of
// 128: 17 beside 335.
#include "attention_plan.h"
#include "attention_short.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"

namespace fpstok {

namespace {

constexpr int kRangeThreads = 256;

struct RangeArgs {
  const __half *dout, *v;
  int64_t do_token, do_head, v_token, v_head;
  int64_t n_q;
  int heads, kv_heads, D;
  const TileItem *queries, *keys, *shorts;
  float* range;  // [2][n_q]: of the event whose first query it is, the largest |dO_i|^2, and |V_j|^2
  const WsHeader* hdr;
};

// The largest sum of squares of a head's `rows` rows (at most kTile), over what
// is finite: another makes its event's gradients what they are whatever the
// scale.  Every load before the first sum.
template <int DP>
__device__ __forceinline__ void largest(const __half* base, int64_t token, int rows, int D, float* to) {
  constexpr int kLanes = DP / 8;  // of a row, 16 bytes each
  constexpr int kAtOnce = kRangeThreads / kLanes, kLoads = kTile / kAtOnce;
  const int c = threadIdx.x % kLanes * 8, row = threadIdx.x / kLanes;
  uint4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    x[i] = row + i * kAtOnce < rows && c < D ? *reinterpret_cast<const uint4*>(base + (row + i * kAtOnce) * token + c)
                                             : make_uint4(0, 0, 0, 0);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack16<__half>(w[k]);
      sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    top = fmaxf(top, sum < INFINITY ? sum : 0.f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  // floats from 0 up are ordered as their bits, and a maximum has no order to depend on
  if ((threadIdx.x & 31) == 0 && top > 0.f) atomicMax(reinterpret_cast<int*>(to), __float_as_int(top));
}

template <int DP>
__global__ void __launch_bounds__(kRangeThreads) k_attn_backward_range(const RangeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_queries = a.hdr->n_items[kQueryTiles], n_keys = a.hdr->n_items[kKeyTiles];
  const int n = n_queries + n_keys + a.hdr->n_items[kShortEvents];
  const auto item = [&](int i) {
    return i < n_queries ? a.queries[i] : i < n_queries + n_keys ? a.keys[i - n_queries] : a.shorts[i - n_queries - n_keys];
  };
  ItemWalk walk(a.heads, n);
  if (!walk.more()) return;
  TileItem e = item(walk.tile), next;
  for (; walk.more(); e = next) {
    const int h = walk.h;
    const bool query = walk.tile < n_queries, key = !query && walk.tile < n_queries + n_keys;
    walk.advance();
    if (walk.more()) next = item(walk.tile);  // on its way while the rows are
    if (e.nq == 0 || e.nk == 0) continue;                                     // no score
    if (key && e.pad[2] != -1 && (e.pad[2] == -2 || e.pad[0] > 0)) continue;  // a tile's second piece, or none
    const int at = query || key ? e.t * kTile : 0;
    if (!key)
      largest<DP>(a.dout + (e.q0 + (int64_t)at) * a.do_token + h * a.do_head, a.do_token, min(kTile, e.nq - at), a.D, a.range + e.q0);
    if (!query && h < a.kv_heads)
      largest<DP>(a.v + (e.k0 + (int64_t)at) * a.v_token + h * a.v_head, a.v_token, min(kTile, e.nk - at), a.D,
                  a.range + a.n_q + e.q0);
  }
}

}  // namespace

cudaError_t launch_attention_backward_range(const AttnCall& c, float* range, const TileItem* queries, const TileItem* keys,
                                            const TileItem* shorts, const WsHeader* hdr, cudaStream_t s) {
  RangeArgs a;
  a.dout = static_cast<const __half*>(c.dout);
  a.v = static_cast<const __half*>(c.v);
  a.do_token = c.do_token;
  a.do_head = c.do_head;
  a.v_token = c.v_token;
  a.v_head = c.v_head;
  a.n_q = c.n_q;
  a.heads = c.heads;
  a.kv_heads = c.kv_heads;
  a.D = c.D;
  a.queries = queries;
  a.keys = keys;
  a.shorts = shorts;
  a.range = range;
  a.hdr = hdr;
  const int64_t items = (max_tiles(c.n_q, c.B) + max_tiles(c.n_kv, c.B)) * c.heads, slots = (int64_t)device_info().sm_count * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < slots ? items : slots));
  cfg.blockDim = dim3(kRangeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, c.D <= 64 ? k_attn_backward_range<64> : k_attn_backward_range<128>, a);
}

}  // namespace fpstok
