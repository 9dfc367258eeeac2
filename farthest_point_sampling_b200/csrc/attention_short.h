// Backward of short events (attention_backward_short.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.h"

namespace fpstok {

struct TileItem;

// What the backward kernels share: the maps of their inputs, and whether
// every gradient row starts on a 32-byte sector and ends on one.
struct BwdMaps {
  CUtensorMap q, k, v, d;
  bool sectors;
};

// -D of the queries that see few keys, into rows[heads + head, query].
cudaError_t launch_attention_backward_rows(const AttnCall& c, float* rows, cudaStream_t s);

// Gradients of the events in `items` (at most 128 queries and 128 keys each),
// and zeros in the gradient rows behind the last event.
cudaError_t launch_attention_backward_short(const AttnCall& c, const BwdMaps& maps, const float* rows,
                                            const TileItem* items, WsHeader* hdr, cudaStream_t s);

}  // namespace fpstok
