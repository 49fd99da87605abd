// Internal interface between the C ABI of the scores (qrita_scores_api.cpp) and
// their kernels (qrita_scores.cu). Not installed; not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qrita.h"
#include "qrita_losses.h"

namespace qrita {

constexpr int kMaxTop = 128;      // alternatives of a row (not above the threads of the smallest block)
constexpr int kMaxScored = 8192;  // given tokens of a row

struct ScoreParams {
  const void* logits;
  int64_t B, V, ld;
  const uint8_t* mask;
  const int32_t* tokens;  // [B, M]
  int M, N;
  Scale c;
  float inv_t, inv_t_lo;  // inv_temperature as a pair
  uint32_t C;             // CTAs per row, and the units of it each of them takes
  int64_t per;
  int group_steps;        // steps of a thread whose largest logit is kept as one
  float* logp;            // [B, M]
  int32_t* rank;
  float* entropy;
  int32_t* top_ids;       // [B, N]
  float* top_logp;
};

int launch_scores(const ScoreParams& prm, int dtype, qrita_stream_t stream);

}  // namespace qrita
