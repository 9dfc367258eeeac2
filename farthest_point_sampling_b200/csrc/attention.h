// Attention over packed events: the call as the kernels see it, and their
// launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fpstok.h"

namespace fpstok {

struct WsHeader;

// Visibility of one event: query i of nq stands at p = i + nk - nq and sees
// key j when p - left <= j <= p + right, or when j < sinks and (not causal or
// j <= p).  Unlimited sides are kFar, beyond every position.
struct AttnMask {
  int causal;
  int left, right;
  int sinks;
};
constexpr int kFar = 1 << 29;

constexpr int kDevWaitTimeout = FPS_DEV_WAIT_TIMEOUT;

// How long a wait for a tile polls, and (tests alone) of which kernels the
// first block leaves its first load out, so that the waits for it run out:
// bits of FPS_SKIP_*.
struct WaitTest {
  int polls, skip;
};

struct AttnCall {
  const void* q;
  const void* k;
  const void* v;
  int dtype;
  int64_t n_q, n_kv;
  int heads, kv_heads, group, D;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  const int64_t* q_offsets;
  const int64_t* kv_offsets;
  int B;
  float scale;
  AttnMask mask;
  int max_tokens;
  int zero_tail;
  WaitTest test;
  void* out;   // [n_q, heads, D]
  float* lse;  // [heads, n_q]
  // backward
  const void* dout;
  int64_t do_token, do_head;
  void* dq;
  void* dk;
  void* dv;
};

// Workspace bytes of a call of these sizes.
size_t attention_forward_bytes(const AttnCall& c);
size_t attention_backward_bytes(const AttnCall& c);
cudaError_t launch_attention_forward(const AttnCall& c, void* workspace, cudaStream_t s);
cudaError_t launch_attention_backward(const AttnCall& c, void* workspace, cudaStream_t s);

}  // namespace fpstok
