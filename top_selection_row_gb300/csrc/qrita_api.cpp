// C ABI of the selection library: argument checks, the delta tables, the
// launch shape, and the host-buffer entry point. See include/qrita.h.

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>

#include <cuda_runtime.h>

#include "qrita.h"
#include "qrita_internal.h"

namespace qrita {
namespace {

// ---------------------------------------------------------------------------
// delta tables (Qrita technical summary, "Methodology", part 1: delta comes
// from precomputed tables derived from the normal quantile function, adapted
// to the target k or p). Phi^-1 is found by bisection on the C library's
// erfc, Phi(z) = erfc(-z / sqrt 2) / 2, to a bracket of 1e-13.
// ---------------------------------------------------------------------------
double normal_cdf(double z) { return 0.5 * std::erfc(-z / std::sqrt(2.0)); }

double normal_quantile(double prob) {
  if (prob <= 0.0) return -std::numeric_limits<double>::infinity();
  if (prob >= 1.0) return std::numeric_limits<double>::infinity();
  double lo = -40.0, hi = 40.0;
  for (int it = 0; it < 200 && hi - lo > 1e-13; ++it) {
    const double mid = 0.5 * (lo + hi);
    if (normal_cdf(mid) < prob) lo = mid;
    else hi = mid;
  }
  return 0.5 * (lo + hi);
}

struct Tables {
  float lut_k[kLutK];
  float lut_p[kLutP];
};

Tables build_tables() {
  Tables t;
  for (int i = 0; i < kLutK; ++i) {
    // Phi^-1(1 - u) = -Phi^-1(u), evaluated in the accurate lower tail
    const double u = std::exp2(-0.25 * i);
    t.lut_k[i] = static_cast<float>(-normal_quantile(u));
  }
  for (int i = 0; i < kLutP; ++i) {
    const double q = std::exp2(-0.25 * i);
    t.lut_p[i] = static_cast<float>(normal_quantile(q));
  }
  return t;
}

const Tables& tables() {
  static const Tables t = build_tables();
  return t;
}

// Truncation tuning (the pages give no constants; these only move speed,
// never the result): u = alpha_k * k / V, truncation skipped above u_max;
// alpha shrinks toward kAlphaMinK when alpha * k survivors would not fit the
// own lists.
constexpr float kAlphaK = 2.0f;
constexpr float kAlphaMinK = 1.25f;
constexpr float kUMaxK = 0.25f;
constexpr float kMarginP = 0.25f;

constexpr int kCtasPerSm = 2;
// Rows shorter than this per CTA are not split further.
constexpr int64_t kMinChunk = 3072;
// Chunk indices must fit below the rank bits of a gathered tag.
constexpr int64_t kMaxChunk = int64_t(1) << 27;

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64 && n > 0) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

int smem_optin() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    int v = cached[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  const int n = max_smem_per_block();
  if (dev >= 0 && dev < 64 && n > 0) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

int elem_bytes(int dtype) { return dtype == QRITA_DTYPE_F32 ? 4 : 2; }

struct Shape {
  int C;
  int chunk;
  int ocap;
  size_t smem;
  bool multi_wave;  // more CTAs than the device holds at once
};

// Rows are reordered (heavy first) only for batches this small: every CTA
// reads all k and p to find its row.
constexpr int64_t kMaxReorderRows = 8192;

// Launch shape: the row is split into C contiguous chunks (one CTA each, one
// cluster per row). C is the largest power of two that keeps the whole batch
// in one wave of resident CTAs, so small batches spread over every SM while
// large batches keep one CTA per row and stream it whole.
int choose_shape(int64_t B, int64_t V, uint32_t flags, Shape* out) {
  const int optin = smem_optin();
  if (optin <= 0) return QRITA_ECUDA;
  int C = 1;
  if (flags & QRITA_FLAG_CLUSTER_SET) {
    const int shift = static_cast<int>((flags >> QRITA_FLAG_CLUSTER_SHIFT) & 7u);
    if (shift > 4) return QRITA_EINVAL;
    C = 1 << shift;
  } else {
    const int64_t slots = static_cast<int64_t>(sm_count()) * kCtasPerSm;
    while (C < kMaxCluster && B * (2 * C) <= slots && (V + 2 * C - 1) / (2 * C) >= kMinChunk) C *= 2;
  }
  while ((V + C - 1) / C > kMaxChunk) {
    if (C >= kMaxCluster) return QRITA_EUNSUPPORTED;
    C *= 2;
  }
  int64_t chunk = (V + C - 1) / C;
  chunk = (chunk + 15) / 16 * 16;
  if (B * C > static_cast<int64_t>(std::numeric_limits<int32_t>::max())) return QRITA_EUNSUPPORTED;
  const int ocap = kOwnCap;
  const size_t smem = smem_bytes(ocap);
  if (smem == 0 || smem > static_cast<size_t>(optin)) return QRITA_EUNSUPPORTED;
  out->multi_wave = B * C > static_cast<int64_t>(sm_count()) * kCtasPerSm;
  out->C = C;
  out->chunk = static_cast<int>(chunk);
  out->ocap = ocap;
  out->smem = smem;
  return QRITA_OK;
}

int check_args(const void* logits, int dtype, int64_t B, int64_t V, const uint8_t* out_mask,
               uint32_t flags) {
  if (dtype != QRITA_DTYPE_F32 && dtype != QRITA_DTYPE_BF16) return QRITA_EINVAL;
  if (B < 0 || V < 1 || V > std::numeric_limits<int32_t>::max()) return QRITA_EINVAL;
  if (flags & ~QRITA_FLAG_KNOWN_MASK) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (logits == nullptr || out_mask == nullptr) return QRITA_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % static_cast<uintptr_t>(elem_bytes(dtype)) != 0)
    return QRITA_EINVAL;
  return QRITA_OK;
}

int select_impl(const void* logits, int dtype, int64_t B, int64_t V, const int32_t* k,
                const float* p, uint8_t* out_mask, qrita_stream_t stream, uint32_t flags,
                int32_t* row_status, qrita_row_info_t* row_info) {
  int rc = check_args(logits, dtype, B, V, out_mask, flags);
  if (rc != QRITA_OK || B == 0) return rc;
  Shape sh;
  rc = choose_shape(B, V, flags, &sh);
  if (rc != QRITA_OK) return rc;
  Params prm;
  std::memset(&prm, 0, sizeof(prm));
  prm.logits = logits;
  prm.mask = out_mask;
  prm.k = k;
  prm.p = p;
  prm.row_status = row_status;
  prm.row_info = row_info;
  prm.B = B;
  prm.V = static_cast<int32_t>(V);
  prm.C = sh.C;
  prm.chunk = sh.chunk;
  prm.ocap = sh.ocap;
  prm.flags = flags;
  prm.heavy_first = (sh.multi_wave && B <= kMaxReorderRows && (p != nullptr || k != nullptr)) ? 1 : 0;
  prm.alpha_k = kAlphaK;
  prm.alpha_min_k = kAlphaMinK;
  prm.margin_p = kMarginP;
  prm.u_max_k = kUMaxK;
  const Tables& t = tables();
  std::memcpy(prm.lut_k, t.lut_k, sizeof(prm.lut_k));
  std::memcpy(prm.lut_p, t.lut_p, sizeof(prm.lut_p));
  const int e = launch_select(prm, dtype, sh.smem, stream);
  return e == 0 ? QRITA_OK : QRITA_ECUDA;
}

dev::F2 pair_of(double v) {
  dev::F2 r;
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
  if (!(inv_temperature > 0.0) || !std::isfinite(inv_temperature)) return QRITA_EINVAL;
  const float c = static_cast<float>(1.4426950408889634074 * inv_temperature);
  if (!std::isfinite(c) || !std::isnormal(c)) return QRITA_EINVAL;
  if (grad != nullptr && ld_grad < V) return QRITA_EINVAL;
  std::memset(out, 0, sizeof(*out));
  out->logits = logits;
  out->B = B;
  out->V = V;
  out->ld = ld;
  out->mask = mask;
  out->tokens = tokens;
  out->c = c;
  const double c_ln2 = static_cast<double>(c) * 0.69314718055994530942;
  out->c_ln2 = static_cast<float>(c_ln2);
  out->c_ln2_lo = static_cast<float>(c_ln2 - out->c_ln2);
  out->inv_t = static_cast<float>(inv_temperature);
  out->inv_b = B > 0 ? static_cast<float>(1.0 / static_cast<double>(B)) : 0.f;
  out->grad = grad;
  out->ld_grad = ld_grad;
  if (B == 0) return QRITA_OK;
  if (logits == nullptr || tokens == nullptr) return QRITA_EINVAL;
  const uint64_t eb = static_cast<uint64_t>(elem_bytes(dtype));
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
    if (!same && x0 < g0 + gn && g0 < x0 + xn) return QRITA_EINVAL;
  }
  return QRITA_OK;
}

size_t align256(size_t x) { return (x + 255u) & ~static_cast<size_t>(255u); }

}  // namespace

int device_sms() { return sm_count(); }

}  // namespace qrita

extern "C" {

int qrita_select(const void* logits, int dtype, int64_t B, int64_t V, const int32_t* k,
                 const float* p, uint8_t* out_mask, qrita_stream_t stream) {
  return qrita::select_impl(logits, dtype, B, V, k, p, out_mask, stream, 0u, nullptr, nullptr);
}

int qrita_select_ex(const void* logits, int dtype, int64_t B, int64_t V, const int32_t* k,
                    const float* p, uint8_t* out_mask, qrita_stream_t stream, uint32_t flags,
                    int32_t* row_status, qrita_row_info_t* row_info) {
  return qrita::select_impl(logits, dtype, B, V, k, p, out_mask, stream, flags, row_status,
                            row_info);
}

size_t qrita_host_staging_bytes(int dtype, int64_t B, int64_t V) {
  if ((dtype != QRITA_DTYPE_F32 && dtype != QRITA_DTYPE_BF16) || B < 0 || V < 1 ||
      V > std::numeric_limits<int32_t>::max())
    return 0;
  // every section and the sum must fit size_t (0 = invalid, as above)
  constexpr size_t kMax = std::numeric_limits<size_t>::max();
  const size_t b = static_cast<size_t>(B), v = static_cast<size_t>(V);
  const size_t eb = static_cast<size_t>(qrita::elem_bytes(dtype));
  if (b != 0 && v > (kMax / 8u) / b) return 0;  // B*V*eb and the 256-byte roundings stay far below kMax
  const size_t n = b * v;
  return qrita::align256(n * eb) + qrita::align256(b * 4) + qrita::align256(b * 4) + qrita::align256(n);
}

int qrita_select_host(const void* h_logits, int dtype, int64_t B, int64_t V, const int32_t* h_k,
                      const float* h_p, uint8_t* h_mask, void* d_staging, size_t staging_bytes,
                      qrita_stream_t stream) {
  int rc = qrita::check_args(h_logits, dtype, B, V, h_mask, 0u);
  if (rc != QRITA_OK || B == 0) return rc;
  const size_t need = qrita_host_staging_bytes(dtype, B, V);
  if (d_staging == nullptr || staging_bytes < need) return QRITA_EINVAL;
  const size_t n = static_cast<size_t>(B) * static_cast<size_t>(V);
  const size_t lb = n * qrita::elem_bytes(dtype);
  unsigned char* base = static_cast<unsigned char*>(d_staging);
  void* d_logits = base;
  int32_t* d_k = reinterpret_cast<int32_t*>(base + qrita::align256(lb));
  float* d_p = reinterpret_cast<float*>(base + qrita::align256(lb) + qrita::align256(B * 4));
  uint8_t* d_mask = base + qrita::align256(lb) + 2 * qrita::align256(B * 4);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // once a copy is enqueued, every return waits for the stream first: the
  // caller may free or reuse its host buffers as soon as the call returns
  auto fail_after_enqueue = [st](int code) {
    (void)cudaStreamSynchronize(st);
    return code;
  };
  if (cudaMemcpyAsync(d_logits, h_logits, lb, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return fail_after_enqueue(QRITA_ECUDA);
  if (h_k && cudaMemcpyAsync(d_k, h_k, B * 4, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return fail_after_enqueue(QRITA_ECUDA);
  if (h_p && cudaMemcpyAsync(d_p, h_p, B * 4, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return fail_after_enqueue(QRITA_ECUDA);
  rc = qrita::select_impl(d_logits, dtype, B, V, h_k ? d_k : nullptr, h_p ? d_p : nullptr, d_mask,
                          stream, 0u, nullptr, nullptr);
  if (rc != QRITA_OK) return fail_after_enqueue(rc);
  if (cudaMemcpyAsync(h_mask, d_mask, n, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return fail_after_enqueue(QRITA_ECUDA);
  if (cudaStreamSynchronize(st) != cudaSuccess) return QRITA_ECUDA;
  return QRITA_OK;
}

int qrita_topk_ids(const void* logits, int dtype, int64_t B, int64_t V, const int32_t* k, int32_t kmax,
                   uint8_t* out_mask, int32_t* out_ids, qrita_stream_t stream) {
  int rc = qrita::check_args(logits, dtype, B, V, out_mask, 0u);
  if (rc != QRITA_OK || B == 0) return rc;
  if (k == nullptr || out_ids == nullptr || kmax < 1 || kmax > qrita::kMaxIds) return QRITA_EINVAL;
  if (B > static_cast<int64_t>(std::numeric_limits<int32_t>::max())) return QRITA_EUNSUPPORTED;
  rc = qrita::select_impl(logits, dtype, B, V, k, nullptr, out_mask, stream, 0u, nullptr, nullptr);
  if (rc != QRITA_OK) return rc;
  return qrita::launch_ids(logits, dtype, B, V, k, kmax, out_mask, out_ids, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_candidates(const void* logits, int dtype, int64_t B, int64_t V, const uint8_t* mask, int32_t cap,
                     int32_t* out_ids, float* out_probs, int32_t* out_count, const float* u, int32_t* out_sample,
                     qrita_stream_t stream) {
  int rc = qrita::check_args(logits, dtype, B, V, mask, 0u);
  if (rc != QRITA_OK || B == 0) return rc;
  if (cap < 1 || out_ids == nullptr || out_probs == nullptr || out_count == nullptr) return QRITA_EINVAL;
  if ((u == nullptr) != (out_sample == nullptr)) return QRITA_EINVAL;
  if (B > static_cast<int64_t>(std::numeric_limits<int32_t>::max())) return QRITA_EUNSUPPORTED;
  return qrita::launch_candidates(logits, dtype, B, V, mask, cap, out_ids, out_probs, out_count, u, out_sample,
                                  stream) == 0
             ? QRITA_OK
             : QRITA_ECUDA;
}

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
  prm.clip_lo = static_cast<float>(1.0 - clip_low);
  prm.clip_hi = static_cast<float>(1.0 + clip_high);
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
  return qrita::launch_policy(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

size_t qrita_preference_workspace_bytes(int64_t B, int64_t P) {
  constexpr int64_t kMax = std::numeric_limits<int32_t>::max();
  if (B < 0 || B > kMax || P < 0 || P > (kMax - 1) / 2) return 0;
  return qrita::pref_workspace_bytes(B, P);
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
  pref.smoothing = label_smoothing;
  pref.margin = margin;
  pref.length_norm = length_norm;
  pref.pair_loss = out_pair_loss;
  pref.log_ratio = out_log_ratio;
  pref.seq_logp = out_seq_logp;
  pref.workspace = workspace;
  return qrita::launch_preference(prm, pref, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_delta_table(int which, float* out, int n) {
  const qrita::Tables& t = qrita::tables();
  const float* src = nullptr;
  int len = 0;
  if (which == 0) {
    src = t.lut_k;
    len = qrita::kLutK;
  } else if (which == 1) {
    src = t.lut_p;
    len = qrita::kLutP;
  } else {
    return -1;
  }
  if (out != nullptr && n > 0) std::memcpy(out, src, sizeof(float) * static_cast<size_t>(n < len ? n : len));
  return len;
}

const char* qrita_strerror(int code) {
  switch (code) {
    case QRITA_OK:
      return "success";
    case QRITA_EINVAL:
      return "invalid argument";
    case QRITA_EUNSUPPORTED:
      return "unsupported size: a row does not fit the shared memory of one cluster";
    case QRITA_ECUDA:
      return "CUDA runtime or launch error";
    default:
      return "unknown error code";
  }
}

int qrita_version(void) { return 200; }

}  // extern "C"
