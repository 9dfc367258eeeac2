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
// A warp per query and head, DP / 8 lanes for a key, 32 / (DP / 8) keys at a
// time, all loads of a query at once: latency bounds it.  Blocks first look for
// the events with such queries, one a thread.  The kernel needs nothing that the
// planning kernel before it writes, and runs beside it.
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
__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
  const uint32_t* px = reinterpret_cast<const uint32_t*>(&x);
  const uint32_t* py = reinterpret_cast<const uint32_t*>(&y);
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 u = unpack16<T>(px[k]), w = unpack16<T>(py[k]);
    s = fmaf(u.x, w.x, fmaf(u.y, w.y, s));
  }
  return s;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kRowThreads) k_attn_backward_rows(const RowArgs a) {
  constexpr int kLanes = DP / 8, kKeys = 32 / kLanes, kSteps = kFewKeys / kKeys;
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, c = (lane % kLanes) * 8, first = lane / kLanes;
  const bool in = c < a.D;
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
      for (int64_t e = blockIdx.y * (kRowThreads / 32) + threadIdx.x / 32; e < (int64_t)end * a.heads;
           e += gridDim.y * (kRowThreads / 32)) {
        const int i = e <= 0x7fffffff ? (int)e / a.heads : (int)(e / a.heads);
        const int h = (int)(e - (int64_t)i * a.heads), g = h / a.group;
        const FewSpan span = row_span(a.mask, i + shift, nk);
        const int n = span.count();
        if (n > kFewKeys) continue;
        const uint4 q = in ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (q0 + i) * a.q_token + h * a.q_head + c) : zero;
        const uint4 d = in ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.dout) + (q0 + i) * a.do_token + h * a.do_head + c) : zero;
        const float lse2 = a.lse[(int64_t)h * a.n_q + q0 + i] * kLog2e;
        uint4 k[kSteps], v[kSteps];
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
          const int key = x * kKeys + first;
          const bool real = in && key < n;
          const int64_t j = k0 + span.key(key);
          k[x] = real ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + j * a.k_token + g * a.k_head + c) : zero;
          v[x] = real ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + j * a.v_token + g * a.v_head + c) : zero;
        }
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
          float s = dot8<T>(q, k[x]), p = dot8<T>(d, v[x]);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            p += __shfl_xor_sync(0xffffffffu, p, o);
          }
          if (x * kKeys + first < n) sum = fmaf(exp2_approx(fmaf(s, a.scale_log2, -lse2)), p, sum);
        }
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) a.rows[((int64_t)a.heads + h) * a.n_q + q0 + i] = -sum;
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
