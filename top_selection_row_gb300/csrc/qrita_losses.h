// Internal interface between the C ABI of the losses (qrita_losses_api.cpp) and
// their kernels (qrita_losses.cu). Not installed; not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qrita.h"

namespace qrita {

// An fp32 value in two parts: hi + lo with |lo| <= ulp(hi)/2.
struct LossPair {
  float hi, lo;
};

// c = log2(e) * inv_temperature, hi + lo: weights are 2^((x - m) c). Logits an
// octave (1 / c) apart differ by a factor of 2 in weight, and one a thousand
// octaves below another (bottom, < 0) has none beside it.
struct Scale {
  float hi, lo, octave, bottom;
};

// Arguments of the loss kernels; null pointers are the optional arguments of
// the C ABI.
struct LossParams {
  const void* logits;
  int64_t B, V, ld;
  const uint8_t* mask;
  const int32_t* tokens;  // [B], or [B, K]
  int K;                  // qrita_token_scores_grad's ids of a row
  Scale c;
  float inv_t, inv_t_lo;  // inv_temperature as a pair
  float inv_b;  // 1 / B
  uint32_t C;   // CTAs per row, and the units of it each of them takes
  int64_t per;
  // outputs per row
  float* logp;
  float* entropy;
  float* kl;
  float* row_loss;
  void* grad;
  int64_t ld_grad;
  const float* grad_loss;
  // qrita_token_logprobs_grad, qrita_token_scores_grad
  const float* g_logp;
  const float* g_entropy;
  // qrita_policy_loss
  const float* old_logp;
  const float* ref_logp;
  const float* advantages;
  const float* weights;
  LossPair clip_lo, clip_hi;  // 1 - clip_low, 1 + clip_high
  LossPair ln_lo, ln_hi;      // their logarithms (-inf, inf: no clip)
  float kl_coef, entropy_coef;
  float* loss;
  bool give_back;  // tensor memory, without waiting for the cluster (tests)
};

constexpr int kMaxGradIds = 256;  // K, at most

struct PrefParams {
  const int32_t* starts;
  int64_t P;
  const float* ref;
  const float* weights;
  double beta, smoothing, margin;
  float beta_parts[2];  // their product is beta, also beyond fp32 (up to 2^253)
  int length_norm;
  float inv_p;  // 1 / P
  float* pair_loss;
  float* log_ratio;
  float* seq_logp;
  void* workspace;
};

size_t pref_workspace_bytes(int64_t B);

// Checks of the arguments that every entry point over rows shares (a QRITA_* code),
// and the row part of *out.
int row_args(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
             const int32_t* tokens, double inv_temperature, void* grad, int64_t ld_grad, LossParams* out);

// Every launch returns a cudaError_t.
int launch_logprobs(const LossParams& prm, int dtype, qrita_stream_t stream);
int launch_logprobs_grad(const LossParams& prm, int dtype, qrita_stream_t stream);
int launch_scores_grad(const LossParams& prm, int dtype, qrita_stream_t stream);
int launch_policy(const LossParams& prm, int dtype, qrita_stream_t stream);
int launch_preference(const LossParams& prm, const PrefParams& pref, int dtype, qrita_stream_t stream);

}  // namespace qrita
