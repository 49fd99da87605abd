// C ABI of the scores over rows of logits: argument checks and the constants the
// kernels take. See include/qrita.h.

#include <cstdint>

#include "qrita.h"
#include "qrita_losses.h"
#include "qrita_scores.h"

extern "C" {

int qrita_token_scores(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                       const int32_t* tokens, int32_t M, int32_t N, double inv_temperature, float* out_logp,
                       int32_t* out_rank, float* out_entropy, int32_t* out_top_ids, float* out_top_logp,
                       qrita_stream_t stream) {
  qrita::LossParams row;
  const int rc = qrita::row_args(logits, dtype, B, V, ld, mask, tokens, inv_temperature, nullptr, 0, &row);
  if (rc != QRITA_OK) return rc;
  if (M < 0 || M > qrita::kMaxScored || N < 0 || N > qrita::kMaxTop) return QRITA_EINVAL;
  if (out_rank != nullptr && M == 0) return QRITA_EINVAL;
  if (M == 0 && N == 0 && out_entropy == nullptr) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (M > 0 && (tokens == nullptr || out_logp == nullptr)) return QRITA_EINVAL;
  if (N > 0 && (out_top_ids == nullptr || out_top_logp == nullptr)) return QRITA_EINVAL;
  qrita::ScoreParams prm = {};
  prm.logits = logits;
  prm.B = B;
  prm.V = V;
  prm.ld = ld;
  prm.mask = mask;
  prm.tokens = tokens;
  prm.M = M;
  prm.N = N;
  prm.c = row.c;
  prm.inv_t = row.inv_t;
  prm.inv_t_lo = row.inv_t_lo;
  prm.logp = out_logp;
  prm.rank = out_rank;
  prm.entropy = out_entropy;
  prm.top_ids = out_top_ids;
  prm.top_logp = out_top_logp;
  return qrita::launch_scores(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_token_scores_grad(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                            const int32_t* ids, int32_t K, double inv_temperature, const float* grad_logp,
                            const float* grad_entropy, void* out_grad, int64_t ld_grad, qrita_stream_t stream) {
  qrita::LossParams prm;
  const int rc = qrita::row_args(logits, dtype, B, V, ld, mask, ids, inv_temperature, out_grad, ld_grad, &prm);
  if (rc != QRITA_OK) return rc;
  if (K < 1 || K > qrita::kMaxGradIds) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (ids == nullptr || out_grad == nullptr || (grad_logp == nullptr && grad_entropy == nullptr)) return QRITA_EINVAL;
  prm.K = K;
  prm.g_logp = grad_logp;
  prm.g_entropy = grad_entropy;
  return qrita::launch_scores_grad(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

}  // extern "C"
