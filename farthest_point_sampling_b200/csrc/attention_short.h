// Backward of short events (attention_backward_short.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.h"

namespace fpstok {

struct TileItem;
struct WsHeader;

// What the backward kernels share: the maps of their inputs, and whether
// every gradient row starts on a 32-byte sector and ends on one.
struct BwdMaps {
  CUtensorMap q, k, v, d;
  bool sectors;
};

// What the products of a float16 backward take of an event's P and dS
// (attention_backward_range.cu): 2^kWeightShift P, and c times that of dS.
constexpr int kWeightShift = 14;

// The part of a work item that says so: c, and what takes both scales back.
template <bool kScaled>
struct ItemScale {
  float c, back;
  __device__ __forceinline__ void set(float c_) {
    c = c_;
    back = 1.f / (c * (1 << kWeightShift));
  }
  static constexpr float kBackP = 1.f / (1 << kWeightShift);  // of P alone
};
template <>
struct ItemScale<false> {
  static constexpr float c = 1.f, back = 1.f, kBackP = 1.f;
  __device__ __forceinline__ void set(float) {}
};

// Into range[0 and 1][an event's first query]: its largest |dO_i|^2 and |V_j|^2.
cudaError_t launch_attention_backward_range(const AttnCall& c, float* range, const TileItem* queries, const TileItem* keys,
                                            const TileItem* shorts, const WsHeader* hdr, cudaStream_t s);

// -D of the queries that see few keys, into rows[heads + head, query].
cudaError_t launch_attention_backward_rows(const AttnCall& c, float* rows, cudaStream_t s);

// Gradients of the events in `items` (at most 128 queries and 128 keys each),
// and zeros in the gradient rows behind the last event.
cudaError_t launch_attention_backward_short(const AttnCall& c, const BwdMaps& maps, const float* rows, const float* range,
                                            const TileItem* items, WsHeader* hdr, cudaStream_t s);

}  // namespace fpstok
