// C ABI of the losses over rows of logits: argument checks and the constants
// the kernels take. See include/qrita.h.

#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include "qrita.h"
#include "qrita_losses.h"

namespace qrita {
namespace {

LossPair pair_of(double v) {
  LossPair r;
  r.hi = static_cast<float>(v);
  r.lo = std::isfinite(r.hi) ? static_cast<float>(v - r.hi) : 0.f;
  return r;
}

// Arguments every loss entry point shares; fills the row part of *out.
int loss_args(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
              const int32_t* tokens, double inv_temperature, void* grad, int64_t ld_grad, LossParams* out) {
  if (dtype != QRITA_DTYPE_F32 && dtype != QRITA_DTYPE_BF16) return QRITA_EINVAL;
  constexpr int64_t kMax = std::numeric_limits<int32_t>::max();
  if (B < 0 || B > kMax || V < 1 || V > kMax || ld < V) return QRITA_EINVAL;
  if (!(inv_temperature >= 1e-30 && inv_temperature <= 1e30)) return QRITA_EINVAL;
  const double c = 1.4426950408889634074 * inv_temperature;
  if (grad != nullptr && ld_grad < V) return QRITA_EINVAL;
  std::memset(out, 0, sizeof(*out));
  out->logits = logits;
  out->B = B;
  out->V = V;
  out->ld = ld;
  out->mask = mask;
  out->tokens = tokens;
  out->c.hi = static_cast<float>(c);
  out->c.lo = static_cast<float>(c - out->c.hi);
  out->c.octave = static_cast<float>(1.0 / c);
  out->c.bottom = static_cast<float>(-1000.0 / c);
  out->inv_t = static_cast<float>(inv_temperature);
  out->inv_t_lo = static_cast<float>(inv_temperature - out->inv_t);
  out->inv_b = B > 0 ? static_cast<float>(1.0 / static_cast<double>(B)) : 0.f;
  out->grad = grad;
  out->ld_grad = ld_grad;
  if (B == 0) return QRITA_OK;
  if (logits == nullptr || tokens == nullptr) return QRITA_EINVAL;
  const uint64_t eb = static_cast<uint64_t>(dtype == QRITA_DTYPE_F32 ? 4 : 2);
  const uint64_t x0 = reinterpret_cast<uintptr_t>(logits), g0 = reinterpret_cast<uintptr_t>(grad);
  if (x0 % eb != 0 || g0 % eb != 0) return QRITA_EINVAL;
  // a row stride whose last byte offset leaves 64 bits is no tensor
  const uint64_t rows = static_cast<uint64_t>(B - 1);
  const uint64_t most = static_cast<uint64_t>(std::numeric_limits<int64_t>::max()) / eb - static_cast<uint64_t>(V);
  if (rows != 0 && static_cast<uint64_t>(ld) > most / rows) return QRITA_EINVAL;
  if (grad != nullptr) {
    if (rows != 0 && static_cast<uint64_t>(ld_grad) > most / rows) return QRITA_EINVAL;
    const uint64_t xn = (rows * static_cast<uint64_t>(ld) + static_cast<uint64_t>(V)) * eb;
    const uint64_t gn = (rows * static_cast<uint64_t>(ld_grad) + static_cast<uint64_t>(V)) * eb;
    const bool same = x0 == g0 && (ld == ld_grad || B == 1);
    // rows side by side in wider ones: apart by [V, ld - V] modulo ld
    bool apart = false;
    if (ld == ld_grad && x0 % eb == g0 % eb) {
      const uint64_t d = (x0 < g0 ? g0 - x0 : x0 - g0) / eb % static_cast<uint64_t>(ld);
      apart = d >= static_cast<uint64_t>(V) && d <= static_cast<uint64_t>(ld - V);
    }
    if (!same && !apart && x0 < g0 + gn && g0 < x0 + xn) return QRITA_EINVAL;
  }
  return QRITA_OK;
}

}  // namespace
}  // namespace qrita

extern "C" {

int qrita_token_logprobs(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                         const int32_t* tokens, double inv_temperature, float* out_logp, float* out_entropy,
                         qrita_stream_t stream) {
  qrita::LossParams prm;
  const int rc = qrita::loss_args(logits, dtype, B, V, ld, mask, tokens, inv_temperature, nullptr, 0, &prm);
  if (rc != QRITA_OK || B == 0) return rc;
  if (out_logp == nullptr) return QRITA_EINVAL;
  prm.logp = out_logp;
  prm.entropy = out_entropy;
  return qrita::launch_logprobs(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_token_logprobs_grad(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                              const int32_t* tokens, double inv_temperature, const float* grad_logp,
                              const float* grad_entropy, void* out_grad, int64_t ld_grad, qrita_stream_t stream) {
  qrita::LossParams prm;
  const int rc = qrita::loss_args(logits, dtype, B, V, ld, mask, tokens, inv_temperature, out_grad, ld_grad, &prm);
  if (rc != QRITA_OK || B == 0) return rc;
  if (out_grad == nullptr || (grad_logp == nullptr && grad_entropy == nullptr)) return QRITA_EINVAL;
  prm.g_logp = grad_logp;
  prm.g_entropy = grad_entropy;
  return qrita::launch_logprobs_grad(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_policy_loss(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                      const int32_t* tokens, double inv_temperature, const float* old_logp, const float* ref_logp,
                      const float* advantages, const float* weights, double clip_low, double clip_high, double kl_coef,
                      double entropy_coef, const float* grad_loss, float* out_loss, float* out_row_loss,
                      float* out_logp, float* out_kl, float* out_entropy, void* out_grad, int64_t ld_grad,
                      qrita_stream_t stream) {
  return qrita_policy_loss_ex(logits, dtype, B, V, ld, mask, tokens, inv_temperature, old_logp, ref_logp, advantages,
                              weights, clip_low, clip_high, kl_coef, entropy_coef, grad_loss, out_loss, out_row_loss,
                              out_logp, out_kl, out_entropy, out_grad, ld_grad, 0u, stream);
}

int qrita_policy_loss_ex(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const uint8_t* mask,
                         const int32_t* tokens, double inv_temperature, const float* old_logp, const float* ref_logp,
                         const float* advantages, const float* weights, double clip_low, double clip_high,
                         double kl_coef, double entropy_coef, const float* grad_loss, float* out_loss,
                         float* out_row_loss, float* out_logp, float* out_kl, float* out_entropy, void* out_grad,
                         int64_t ld_grad, uint32_t flags, qrita_stream_t stream) {
  if ((flags & ~QRITA_LOSS_FLAG_TEST_GIVE_BACK) != 0u) return QRITA_EINVAL;
  qrita::LossParams prm;
  const int rc = qrita::loss_args(logits, dtype, B, V, ld, mask, tokens, inv_temperature, out_grad, ld_grad, &prm);
  if (rc != QRITA_OK) return rc;
  if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0)) return QRITA_EINVAL;
  if (!(kl_coef >= 0.0) || !std::isfinite(static_cast<float>(kl_coef)) ||
      !std::isfinite(static_cast<float>(entropy_coef)))
    return QRITA_EINVAL;
  if (out_loss == nullptr) return QRITA_EINVAL;
  if (B > 0 && (advantages == nullptr || out_row_loss == nullptr)) return QRITA_EINVAL;
  prm.old_logp = old_logp;
  prm.ref_logp = ref_logp;
  prm.advantages = advantages;
  prm.weights = weights;
  prm.clip_lo = qrita::pair_of(1.0 - clip_low);
  prm.clip_hi = qrita::pair_of(1.0 + clip_high);
  prm.ln_lo = qrita::pair_of(std::log(1.0 - clip_low));
  prm.ln_hi = qrita::pair_of(std::log1p(clip_high));
  prm.kl_coef = static_cast<float>(kl_coef);
  prm.entropy_coef = static_cast<float>(entropy_coef);
  prm.grad_loss = grad_loss;
  prm.loss = out_loss;
  prm.row_loss = out_row_loss;
  prm.logp = out_logp;
  prm.kl = out_kl;
  prm.entropy = out_entropy;
  prm.give_back = (flags & QRITA_LOSS_FLAG_TEST_GIVE_BACK) != 0u;
  return qrita::launch_policy(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

size_t qrita_preference_workspace_bytes(int64_t B, int64_t P) {
  constexpr int64_t kMax = std::numeric_limits<int32_t>::max();
  if (B < 0 || B > kMax || P < 0 || P > (kMax - 1) / 2) return 0;
  return qrita::pref_workspace_bytes(B);
}

int qrita_preference_loss(const void* logits, int dtype, int64_t B, int64_t V, int64_t ld, const int32_t* tokens,
                          double inv_temperature, const int32_t* starts, int64_t P, const float* ref_logp,
                          const float* weights, double beta, double label_smoothing, double margin, int length_norm,
                          const float* grad_loss, float* out_loss, float* out_pair_loss, float* out_log_ratio,
                          float* out_seq_logp, float* out_logp, void* out_grad, int64_t ld_grad, void* workspace,
                          size_t workspace_bytes, qrita_stream_t stream) {
  qrita::LossParams prm;
  const int rc = qrita::loss_args(logits, dtype, B, V, ld, nullptr, tokens, inv_temperature, out_grad, ld_grad, &prm);
  if (rc != QRITA_OK) return rc;
  if (!(beta > 0.0) || !std::isfinite(beta) || !std::isfinite(margin)) return QRITA_EINVAL;
  if (!(label_smoothing >= 0.0 && label_smoothing <= 1.0)) return QRITA_EINVAL;
  if (length_norm != 0 && length_norm != 1) return QRITA_EINVAL;
  const size_t need = qrita_preference_workspace_bytes(B, P);
  if (need == 0 || out_loss == nullptr) return QRITA_EINVAL;
  if (P > 0 && (starts == nullptr || out_pair_loss == nullptr || out_log_ratio == nullptr || out_seq_logp == nullptr))
    return QRITA_EINVAL;
  if (workspace == nullptr || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16u != 0)
    return QRITA_EINVAL;
  prm.grad_loss = grad_loss;
  prm.loss = out_loss;
  prm.logp = out_logp;
  qrita::PrefParams pref;
  pref.starts = starts;
  pref.P = P;
  pref.ref = ref_logp;
  pref.weights = weights;
  pref.beta = beta;
  pref.beta_parts[1] = beta > 0x1p126 ? 0x1p126f : 1.f;
  pref.beta_parts[0] = static_cast<float>(std::fmin(beta / pref.beta_parts[1], 0x1p127));
  pref.smoothing = label_smoothing;
  pref.margin = margin;
  pref.length_norm = length_norm;
  pref.pair_loss = out_pair_loss;
  pref.log_ratio = out_log_ratio;
  pref.seq_logp = out_seq_logp;
  pref.workspace = workspace;
  return qrita::launch_preference(prm, pref, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

}  // extern "C"
