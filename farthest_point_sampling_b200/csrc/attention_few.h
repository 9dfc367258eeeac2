// Attention of events with few query rows (attention_few.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace fpstok {

struct TileItem;
struct WsHeader;

constexpr int kFewRows = 16;  // query rows (queries of an event times the heads of a group) of one tile

// One event cut into several chunks.
struct JoinItem {
  int q0, nq, slot, chunks;  // first partial result's slot
};

struct FewPlan {
  int chunk;             // keys of one
  const TileItem* units; // (event, chunk); pad[0] = chunks of the event, pad[1] = its first slot
  const JoinItem* joins;
  float* partial;        // few_partial_floats()
};

// Keys of one chunk for a call of these sizes.
int few_chunk(int64_t n_kv, int kv_heads);
size_t few_partial_floats(int64_t n_kv, int kv_heads, int D, int chunk);
cudaError_t launch_attention_few(const AttnCall& c, const FewPlan& plan, WsHeader* hdr, cudaStream_t s);

}  // namespace fpstok
