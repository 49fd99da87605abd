// Internal interface between the C ABI of the key-value cache's entry points
// (qrita_cache_api.cpp) and their kernels (qrita_cache.cu). Not installed; not part
// of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qrita.h"

namespace qrita {

// Rows of bytes in a [B, H, slots] tensor: strides in bytes.
struct CacheRows {
  void* at;
  int64_t bytes;  // of a row
  int64_t batch, head, slot;
};

// What a cache's slots are ordered by, [B, H, S] and [B].
struct CacheOrder {
  int64_t B, H, S;
  float* weights;
  int32_t* positions;  // null: a slot is its token's position
  int32_t* lengths;
  int32_t* seen;       // null: lengths
  int32_t budget, sink, recent;
};

struct WeightParams {
  CacheOrder c;
  const void* query;
  int64_t q_batch, q_token, q_head;  // strides, elements
  const void* keys;
  int64_t k_batch, k_head, k_slot;
  int32_t G, T, D;
  float scale, decay;
  uint32_t flags;    // QRITA_CACHE_FLAG_*
  int32_t rows;      // query rows a CTA has at once
  int32_t stash;     // floats of a row of kept scores (0: scores are worked out twice)
};

struct EvictParams {
  CacheOrder c;
  CacheRows key, value, out_key, out_value;
  int64_t out_slots_of;  // slots of a row of out_weights and out_positions
  float* out_weights;
  int32_t* out_positions;
  int32_t* out_slots;    // [B, H, budget]
  int32_t* out_lengths;
  int32_t share;         // weights a CTA of the selection keeps in shared memory (0: none)
  bool give_up;          // tests: the bounded waits for bulk copies do so at once
};

struct InsertParams {
  CacheOrder c;
  CacheRows key, value, new_key, new_value;
  int32_t* out_slots;  // [B, H]
};

// Launches qrita_cache_window.cu's kernel (bf16 rows of 16-byte units on their
// boundaries; *result is a cudaError_t), or returns false where its sizes and strides
// are none that it takes.
bool launch_cache_window(const WeightParams& prm, qrita_stream_t stream, int* result);

// Every launch returns a cudaError_t.
int launch_cache_weights(const WeightParams& prm, int dtype, qrita_stream_t stream);
int launch_cache_evict(const EvictParams& prm, qrita_stream_t stream);
int launch_cache_insert(const InsertParams& prm, qrita_stream_t stream);

}  // namespace qrita
