// Attention over packed events, one warp per row: the plain form of every
// case, forward and backward.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

namespace fpstok {

namespace {

constexpr int kRowWarps = 4;

template <typename T>
__device__ __forceinline__ float ld(const T* p);
template <>
__device__ __forceinline__ float ld<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float ld<__half>(const __half* p) { return __half2float(*p); }
template <typename T>
__device__ __forceinline__ void st(T* p, float v);
template <>
__device__ __forceinline__ void st<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ void st<__half>(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ bool sees(const AttnMask& m, int64_t p, int64_t j) {
  const int64_t d = p > j ? p - j : j - p;
  return (m.window < 0 || d <= m.window || j < m.sinks) && (!m.causal || j <= p);
}

// The event holding row r, or -1 (rows behind the last event, or bad offsets).
__device__ __forceinline__ int event_of(const int64_t* off, int B, int64_t r) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (off[m + 1] > r) hi = m; else lo = m + 1;
  }
  return lo < B && off[lo] <= r ? lo : -1;
}

struct Span {
  int64_t q0, k0;
  int64_t nq, nk;
  bool ok;
};
__device__ __forceinline__ Span span_of(const AttnCall& c, int b, WsHeader* hdr) {
  Span s;
  s.q0 = c.q_offsets[b];
  s.k0 = c.kv_offsets[b];
  s.nq = c.q_offsets[b + 1] - s.q0;
  s.nk = c.kv_offsets[b + 1] - s.k0;
  s.ok = s.q0 >= 0 && s.k0 >= 0 && s.nq >= 0 && s.nk >= 0 && s.q0 + s.nq <= c.n_q && s.k0 + s.nk <= c.n_kv;
  if (!s.ok) record_error(hdr, kDevBadOffsets);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// dq of one (query, head); delta recomputed where needed.
template <typename T>
__global__ void k_attn_row_dq(const AttnCall c, WsHeader* hdr) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (w >= c.n_q * c.heads) return;
  const int64_t r = w / c.heads;
  const int h = (int)(w - r * c.heads);
  T* dq = static_cast<T*>(c.dq) + (r * c.heads + h) * c.D;
  const int b = event_of(c.q_offsets, c.B, r);
  Span sp;
  if (b >= 0) sp = span_of(c, b, hdr);
  float qv[4], dov[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (b >= 0 && sp.ok) {
    const T* q = static_cast<const T*>(c.q) + r * c.q_token + h * c.q_head;
    const T* go = static_cast<const T*>(c.dout) + r * c.do_token + h * c.do_head;
    const T* o = static_cast<const T*>(c.out) + (r * c.heads + h) * c.D;
    const int64_t p = r - sp.q0 + sp.nk - sp.nq;
    const float lse = c.lse[(int64_t)h * c.n_q + r];
    float delta = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = lane + 32 * i < c.D;
      qv[i] = in ? ld(q + lane + 32 * i) * c.scale : 0.f;
      dov[i] = in ? ld(go + lane + 32 * i) : 0.f;
      if (in) delta = fmaf(dov[i], ld(o + lane + 32 * i), delta);
    }
    delta = warp_sum(delta);
    for (int64_t j = 0; j < sp.nk; ++j) {
      if (!sees(c.mask, p, j)) continue;
      const T* k = static_cast<const T*>(c.k) + (sp.k0 + j) * c.k_token + (h / c.group) * c.k_head;
      const T* v = static_cast<const T*>(c.v) + (sp.k0 + j) * c.v_token + (h / c.group) * c.v_head;
      float s = 0.f, dp = 0.f, kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < c.D) {
          kv[i] = ld(k + lane + 32 * i);
          s = fmaf(qv[i], kv[i], s);
          dp = fmaf(dov[i], ld(v + lane + 32 * i), dp);
        }
      s = warp_sum(s);
      dp = warp_sum(dp);
      const float ds = expf(s - lse) * (dp - delta);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < c.D) acc[i] = fmaf(ds, kv[i], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < c.D) st(dq + lane + 32 * i, acc[i] * c.scale);
}

// dk, dv of one (key, kv head): the queries of every head that shares it.
template <typename T>
__global__ void k_attn_row_dkv(const AttnCall c, WsHeader* hdr) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (w >= c.n_kv * c.kv_heads) return;
  const int64_t r = w / c.kv_heads;
  const int g = (int)(w - r * c.kv_heads);
  T* dk = static_cast<T*>(c.dk) + (r * c.kv_heads + g) * c.D;
  T* dv = static_cast<T*>(c.dv) + (r * c.kv_heads + g) * c.D;
  const int b = event_of(c.kv_offsets, c.B, r);
  Span sp;
  if (b >= 0) sp = span_of(c, b, hdr);
  float ak[4] = {0.f, 0.f, 0.f, 0.f}, av[4] = {0.f, 0.f, 0.f, 0.f};
  if (b >= 0 && sp.ok) {
    const T* k = static_cast<const T*>(c.k) + r * c.k_token + g * c.k_head;
    const T* v = static_cast<const T*>(c.v) + r * c.v_token + g * c.v_head;
    const int64_t j = r - sp.k0;
    float kv[4], vv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kv[i] = lane + 32 * i < c.D ? ld(k + lane + 32 * i) * c.scale : 0.f;
      vv[i] = lane + 32 * i < c.D ? ld(v + lane + 32 * i) : 0.f;
    }
    for (int64_t i0 = 0; i0 < sp.nq; ++i0) {
      if (!sees(c.mask, i0 + sp.nk - sp.nq, j)) continue;
      for (int h = g * c.group; h < (g + 1) * c.group; ++h) {
        const int64_t qr = sp.q0 + i0;
        const T* q = static_cast<const T*>(c.q) + qr * c.q_token + h * c.q_head;
        const T* go = static_cast<const T*>(c.dout) + qr * c.do_token + h * c.do_head;
        const T* o = static_cast<const T*>(c.out) + (qr * c.heads + h) * c.D;
        float s = 0.f, dp = 0.f, delta = 0.f, qv[4], dov[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < c.D) {
            qv[i] = ld(q + lane + 32 * i);
            dov[i] = ld(go + lane + 32 * i);
            s = fmaf(qv[i], kv[i], s);
            dp = fmaf(dov[i], vv[i], dp);
            delta = fmaf(dov[i], ld(o + lane + 32 * i), delta);
          }
        s = warp_sum(s);
        dp = warp_sum(dp);
        delta = warp_sum(delta);
        const float pr = expf(s - c.lse[(int64_t)h * c.n_q + qr]);
        const float ds = pr * (dp - delta);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < c.D) {
            ak[i] = fmaf(ds, qv[i], ak[i]);
            av[i] = fmaf(pr, dov[i], av[i]);
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < c.D) {
      st(dk + lane + 32 * i, ak[i] * c.scale);
      st(dv + lane + 32 * i, av[i]);
    }
}

// Every event's offsets, and its length against max_tokens.
__global__ void k_attn_check(const AttnCall c, WsHeader* hdr) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= c.B) return;
  if (b == 0 && (c.q_offsets[0] != 0 || c.kv_offsets[0] != 0)) record_error(hdr, kDevBadOffsets);
  const Span sp = span_of(c, b, hdr);
  if (sp.ok && c.max_tokens > 0 && (sp.nq > c.max_tokens || sp.nk > c.max_tokens)) record_error(hdr, kDevTooLarge);
}

cudaError_t check(const AttnCall& c, WsHeader* hdr, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(hdr, 0, sizeof(WsHeader), s);
  if (e != cudaSuccess || c.B == 0) return e;
  count_launch();
  k_attn_check<<<(c.B + 255) / 256, 256, 0, s>>>(c, hdr);
  return cudaGetLastError();
}

unsigned row_blocks(int64_t rows) { return (unsigned)((rows + kRowWarps - 1) / kRowWarps); }

}  // namespace

size_t attention_workspace_bytes(int64_t n_q, int64_t, int B, int, int, int, bool) { return attention_forward_bytes(n_q, B); }

cudaError_t launch_attention(const AttnCall& c, void* workspace, cudaStream_t s) {
  return launch_attention_forward(c, workspace, s);
}

cudaError_t launch_attention_backward(const AttnCall& c, void* workspace, cudaStream_t s) {
  WsHeader* hdr = static_cast<WsHeader*>(workspace);
  cudaError_t e = check(c, hdr, s);
  if (e != cudaSuccess) return e;
  const bool bf = c.dtype == FPS_DTYPE_BF16;
  if (c.n_q) {
    count_launch();
    if (bf) k_attn_row_dq<__nv_bfloat16><<<row_blocks(c.n_q * c.heads), 32 * kRowWarps, 0, s>>>(c, hdr);
    else k_attn_row_dq<__half><<<row_blocks(c.n_q * c.heads), 32 * kRowWarps, 0, s>>>(c, hdr);
  }
  if (c.n_kv) {
    count_launch();
    if (bf) k_attn_row_dkv<__nv_bfloat16><<<row_blocks(c.n_kv * c.kv_heads), 32 * kRowWarps, 0, s>>>(c, hdr);
    else k_attn_row_dkv<__half><<<row_blocks(c.n_kv * c.kv_heads), 32 * kRowWarps, 0, s>>>(c, hdr);
  }
  return cudaGetLastError();
}

}  // namespace fpstok
