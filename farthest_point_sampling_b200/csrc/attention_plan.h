// The tile lists of an attention call, and the tensor maps of its inputs.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.h"

namespace fpstok {

struct TileItem;
struct JoinItem;

// WsHeader::n_items of the lists.
constexpr int kQueryTiles = 0;
constexpr int kKeyTiles = 1;
constexpr int kFewUnits = 2;
constexpr int kFewJoins = 3;
constexpr int kShortEvents = 4;
constexpr int kKeySlots = 5;

// 16-bit rows that a call writes for its queries or its keys: up to two
// tensors of `values` a row (a multiple of 8), and a float for each of `heads`.
struct PlanRows {
  void* rows[2];
  int64_t values;
  float* lse;
  int heads;
};

// The lists of one call; those that are NULL are not made.
struct PlanLists {
  TileItem* queries;  // tiles of 128 queries
  TileItem* keys;     // tiles of 128 keys
  TileItem* units;    // chunks of the events with at most kFewRows query rows, which then have no query tiles
  JoinItem* joins;    // those of them with several chunks
  int chunk;
  // Key tiles that every query sees take the work of a whole event: those of
  // more than `piece` (0: none) streamed tiles of `stream` rows are cut into
  // pieces, pad[0] .. pad[1] - 1 of the tiles of all heads in turn, whose sums
  // go to slot pad[2] (-1: to the gradients; -2: a piece that is not needed).
  int piece, stream, slots;
  JoinItem* key_joins;  // per slot: at a tile's first one its rows and how many, else none
  TileItem* shorts;   // the events of at most 128 queries and 128 keys, which then have no tiles of either kind
  PlanRows of_queries, of_keys;  // what the call writes
  float* range;  // [2][n_q]: set to 0 at every event's first query
};

// Fills the lists, 1024 events at a time and long ones of these first, their
// counts in hdr->n_items, and resets the call's status words.  An event longer
// than max_tokens is recorded and is in no list; inconsistent offsets are
// recorded and end the lists before the 1024 events they are among.  What the
// call would have written for the events in no list is set to NaN.
cudaError_t launch_attention_plan(const AttnCall& c, WsHeader* hdr, const PlanLists& lists, cudaStream_t s);

// Map of a [rows, heads, D] 16-bit tensor for boxes of 64 rows x one head x
// 64 values, 128-byte swizzled; what lies outside reads as zeros.
bool attention_map(CUtensorMap* map, const void* base, bool bf16, int64_t rows, int heads, int D, int64_t token_stride,
                   int64_t head_stride);

// Dynamic shared memory of a kernel above the default limit: set on its first
// launch on each device.
cudaError_t allow_shared_memory(const void* kernel, int bytes);

}  // namespace fpstok
