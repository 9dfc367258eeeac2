// Attention of packed events, backward: D of the queries that see few keys.
//
// D_i = sum_d dO_id O_id of an output that is rounded to 16 bits is off by
// about eps |dO| / sqrt(n) for a query that sees n keys, and with
// dS_ij = P_ij (dP_ij - D_i) that moves its row of dQ by eps / sqrt(n - 1) of
// it: as much as the rounding of dS and of dQ themselves at n = 2, a quarter
// of it at 16; at n = 1, where dS is 0, it is all there is.  So up to kFewKeys
// = 16 keys D is formed from what it stands for,
//   D_i = sum_j P_ij dP_ij,  P_ij = exp(scale q_i k_j - lse_i),  dP_ij = dO_i v_j,
// in float32.  Causal events' first rows, events of a few tokens and narrow
// windows have such queries; over 64 track events of up to 20000 tokens (causal
// window of 511, fp16) the error of dQ and dK falls from 3.2 to 3.0e-4.
//
// A warp takes 16 queries of a head and the keys that those of them with few
// see together (sinks, then at most 31 in a window), 8 at a time, with mma.sync.
// Blocks first look for the events with such queries, one a thread.  The kernel
// needs nothing that the planning kernel before it writes, and runs beside it.
// Where all queries are such, 800000 tokens of 8 heads of 64 in 8 events under a
// window of 4, it takes 0.8 of the backward's 3.4 ms (with a warp per query on
// the CUDA cores 4.9 of 7.5); 2048 events of up to 128 tokens, 12 heads, beside the
// plan: 17 us, and 742 for the gradients.
#include <type_traits>

#include "attention_short.h"
#include "attention_tiles.cuh"
#include "common.cuh"
#include "internal.h"

namespace fpstok {

namespace {

constexpr int kRowThreads = 256;

struct RowArgs {
  const void *q, *k, *v, *dout;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, do_token, do_head;
  const int64_t *q_offsets, *kv_offsets;
  int64_t n_q, n_kv;
  int B, heads, group, D;
  float scale_log2;
  AttnMask mask;
  const float* lse;
  float* rows;
};

struct Event {
  int64_t q0, k0;
  int nk, shift, end;  // keys, position of query 0, queries to look at
};

template <typename T>
__device__ __forceinline__ uint4 load16(const void* base, int64_t at) {
  return *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
}

template <typename T, int DP>
__global__ void __launch_bounds__(kRowThreads) k_attn_backward_rows(const RowArgs a) {
  constexpr int kSpans = DP / 32;
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  __shared__ Event s_event[kRowThreads];
  __shared__ int s_count;
  for (int64_t b0 = blockIdx.x; b0 < a.B; b0 += (int64_t)gridDim.x * kRowThreads) {
    if (threadIdx.x == 0) s_count = 0;
    __syncthreads();
    // an event a thread: those with such queries
    const int64_t b = b0 + (int64_t)gridDim.x * threadIdx.x;
    if (b < a.B) {
      const int64_t q0 = a.q_offsets[b], q1 = a.q_offsets[b + 1], k0 = a.kv_offsets[b], k1 = a.kv_offsets[b + 1];
      // bad offsets are reported by the plan, which leaves the event out
      if (q0 >= 0 && k0 >= 0 && q1 >= q0 && k1 >= k0 && q1 <= a.n_q && k1 <= a.n_kv) {
        const int nq = (int)(q1 - q0), nk = (int)(k1 - k0);
        // but for few keys or a narrow window: positions before the first key,
        // and the first ones of a causal event
        const int end = nk <= kFewKeys || a.mask.left < kFewKeys
                            ? nq
                            : min(nq, max((a.mask.causal ? kFewKeys : 0) - (nk - nq), 0));
        if (end > 0) s_event[atomicAdd(&s_count, 1)] = Event{q0, k0, nk, nk - nq, end};
      }
    }
    __syncthreads();
    for (int n_event = 0; n_event < s_count; ++n_event) {
      const auto [q0, k0, nk, shift, end] = s_event[n_event];
      const int64_t items = (int64_t)((end + 15) / 16) * a.heads;
      for (int64_t e = blockIdx.y * (kRowThreads / 32) + threadIdx.x / 32; e < items; e += gridDim.y * (kRowThreads / 32)) {
        const int tile = e <= 0x7fffffff ? (int)e / a.heads : (int)(e / a.heads);
        const int h = (int)(e - (int64_t)tile * a.heads), i0 = tile * 16;
        // a lane a query: what it sees, and what those with few keys see together
        const int i = i0 + (lane & 15);
        FewSpan span = row_span(a.mask, i + shift, nk);
        const bool few = i < end && span.count() <= kFewKeys;
        if (!few) span = FewSpan{0, 0, 0};
        const uint32_t some = __ballot_sync(kFull, few);
        if (!some) continue;
        const bool in_window = span.hi > span.lo;
        const int s = __reduce_max_sync(kFull, span.s), lo = __reduce_min_sync(kFull, in_window ? span.lo : 0x7fffffff),
                  hi = __reduce_max_sync(kFull, in_window ? span.hi : 0);
        FewSpan mine[2];  // of this thread's two queries
        uint4 q[2][kSpans], d[2][kSpans];
        float lse2[2], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int at = g + 8 * r;
          const bool real = some >> at & 1;
          mine[r].s = __shfl_sync(kFull, span.s, at);
          mine[r].lo = __shfl_sync(kFull, span.lo, at);
          mine[r].hi = __shfl_sync(kFull, span.hi, at);
          const int64_t row = q0 + i0 + at;
#pragma unroll
          for (int x = 0; x < kSpans; ++x) {
            const int c = x * 32 + t * 8;
            q[r][x] = real && c < a.D ? load16<T>(a.q, row * a.q_token + h * a.q_head + c) : zero;
            d[r][x] = real && c < a.D ? load16<T>(a.dout, row * a.do_token + h * a.do_head + c) : zero;
          }
          lse2[r] = real ? a.lse[(int64_t)h * a.n_q + row] * kLog2e : 0.f;
        }
        const int sinks = (s + 7) / 8, blocks = sinks + (hi > lo ? (hi - lo + 7) / 8 : 0);
#pragma unroll 2
        for (int x = 0; x < blocks; ++x) {
          const bool sink = x < sinks;
          const int base = sink ? x * 8 : lo + (x - sinks) * 8, key = base + g;
          const bool real = key < (sink ? s : hi);
          const int64_t row = k0 + key;
          const int head = h / a.group;
          float sc[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int y = 0; y < kSpans; ++y) {
            const int c = y * 32 + t * 8;
            const uint4 k = real && c < a.D ? load16<T>(a.k, row * a.k_token + head * a.k_head + c) : zero;
            const uint4 v = real && c < a.D ? load16<T>(a.v, row * a.v_token + head * a.v_head + c) : zero;
            // a thread's 8 values of a row are those of two products, in any order
            // of the sum that is the same on both sides
            const uint32_t q_lo[4] = {q[0][y].x, q[1][y].x, q[0][y].y, q[1][y].y}, k_lo[2] = {k.x, k.y};
            const uint32_t q_hi[4] = {q[0][y].z, q[1][y].z, q[0][y].w, q[1][y].w}, k_hi[2] = {k.z, k.w};
            const uint32_t d_lo[4] = {d[0][y].x, d[1][y].x, d[0][y].y, d[1][y].y}, v_lo[2] = {v.x, v.y};
            const uint32_t d_hi[4] = {d[0][y].z, d[1][y].z, d[0][y].w, d[1][y].w}, v_hi[2] = {v.z, v.w};
            mma16<T>(sc, q_lo, k_lo);
            mma16<T>(dp, d_lo, v_lo);
            mma16<T>(sc, q_hi, k_hi);
            mma16<T>(dp, d_hi, v_hi);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = base + 2 * t + (c & 1), r = c >> 1;
            const bool seen = sink ? j < mine[r].s : j >= mine[r].lo && j < mine[r].hi;
            if (seen) sum[r] = fmaf(exp2_approx(fmaf(sc[c], a.scale_log2, -lse2[r])), dp[c], sum[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[r] += __shfl_xor_sync(kFull, sum[r], 1);
          sum[r] += __shfl_xor_sync(kFull, sum[r], 2);
          if (t == 0 && (some >> (g + 8 * r) & 1)) a.rows[((int64_t)a.heads + h) * a.n_q + q0 + i0 + g + 8 * r] = -sum[r];
        }
      }
    }
    __syncthreads();
  }
  // the kernels after this one wait for it, and with this for the plan
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T>
cudaError_t run(const RowArgs& a, cudaStream_t s) {
  const auto kernel = a.D <= 64 ? k_attn_backward_rows<T, 64> : k_attn_backward_rows<T, 128>;
  // the events over an SM's worth of blocks each, their queries over the rest
  const int sms = device_info().sm_count, x = a.B < 1 ? 1 : a.B < sms ? a.B : sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)x, (unsigned)(sms * 8 / x));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_attention_backward_rows(const AttnCall& c, float* rows, cudaStream_t s) {
  RowArgs a;
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.dout = c.dout;
  a.q_token = c.q_token;
  a.q_head = c.q_head;
  a.k_token = c.k_token;
  a.k_head = c.k_head;
  a.v_token = c.v_token;
  a.v_head = c.v_head;
  a.do_token = c.do_token;
  a.do_head = c.do_head;
  a.q_offsets = c.q_offsets;
  a.kv_offsets = c.kv_offsets;
  a.n_q = c.n_q;
  a.n_kv = c.n_kv;
  a.B = c.B;
  a.heads = c.heads;
  a.group = c.group;
  a.D = c.D;
  a.scale_log2 = c.scale * kLog2e;
  a.mask = c.mask;
  a.lse = c.lse;
  a.rows = rows;
  return c.dtype == FPS_DTYPE_BF16 ? run<__nv_bfloat16>(a, s) : run<__half>(a, s);
}

}  // namespace fpstok
