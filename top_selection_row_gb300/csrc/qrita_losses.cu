// Losses over rows of logits and their gradients: log-probabilities of given
// tokens, the clipped policy loss with a KL term, and the preference loss on
// paired sequences.
//
// Qrita technical summary (gist.science, paper 2602.01518), "Problem
// statement": the candidate set and the drawn token feed reinforcement
// learning; these kernels score the drawn tokens under the same logits (and
// the same keep-mask).
//
// Everything is in base 2. With c = log2(e) * inv_temperature and m the
// largest kept logit, a kept logit weighs e_j = 2^y_j, y_j = (x_j - m) c, and
//   S = sum e_j,  T = sum e_j y_j,
//   logp_t = ln2 (y_t - log2 S),  H = ln2 (log2 S - T / S),  p_j = e_j / S.
// The difference x_j - m comes before the product, so rows of the type's
// lowest value (a common way to mask) keep their uniform softmax. Every
// gradient here has the form
//   g_j = a dlogp_t/dx_j + h dH/dx_j
//       = inv_t (a [j = t] - p_j (a + h (log p_j + H)))
//       = e_j (A + Hc y_j)     for j != t,
// with A = -inv_t (a + h (H - ln S)) / S and Hc = -inv_t h ln2 / S; the
// token's own entry is written from a (1 - p_t) by expm1, which keeps its
// digits when p_t is near 1.

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "qrita_device.cuh"
#include "qrita_internal.h"

namespace qrita {
namespace {

using namespace dev;

constexpr int kLossThreads = 256;
constexpr int kLossWarps = kLossThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;
constexpr double kLn2 = 0.69314718055994530942;
// Exponents below this give weights of 0 in fp32; the clamp keeps products
// of such a weight with its exponent (an entropy's terms) from being 0 * inf.
constexpr float kMinExp = -1000.0f;

// What a pass computes for a row.
enum class Op { kLogprobs, kGrad, kPolicy, kPrefStats };

// Partial softmax sums of some of a row's logits: their maximum, S and T
// relative to it (-inf and 0 before the first kept logit).
struct Stat {
  float m, s, t;
};

// g_j = 2^y_j (a + h y_j), y_j = (x_j - m) c; the token's own entry is `at`.
struct RowGrad {
  float m, a, h, at;
};

// Per-row record of the preference loss between its kernels.
struct RowStat {
  double logp;
  float m;
  float s;  // below 0: the row joins nothing
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* row, int64_t j) {
  if constexpr (DT == QRITA_DTYPE_F32) {
    return static_cast<const float*>(row)[j];
  } else {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short*>(row)[j]) << 16);
  }
}

template <int DT>
__device__ __forceinline__ void store_grad(void* row, int64_t j, float g) {
  if constexpr (DT == QRITA_DTYPE_F32) {
    static_cast<float*>(row)[j] = g;
  } else {
    // the one rounding of a bf16 gradient, to nearest even
    unsigned short b;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(g));
    static_cast<unsigned short*>(row)[j] = b;
  }
}

template <int DT>
__device__ __forceinline__ const void* row_at(const void* base, int64_t row, int64_t ld) {
  return static_cast<const unsigned char*>(base) + row * ld * (DT == QRITA_DTYPE_F32 ? 4 : 2);
}

template <int DT>
__device__ __forceinline__ void* row_at(void* base, int64_t row, int64_t ld) {
  return static_cast<unsigned char*>(base) + row * ld * (DT == QRITA_DTYPE_F32 ? 4 : 2);
}

// The sums relative to the larger of two maxima.
template <bool ENT>
__device__ __forceinline__ Stat stat_merge(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  // (a maximum of -inf comes with sums of 0, which any finite shift leaves 0)
  const float da = a.m == m ? 0.f : fmaxf((a.m - m) * c, kMinExp);
  const float db = b.m == m ? 0.f : fmaxf((b.m - m) * c, kMinExp);
  const float fa = ex2(da), fb = ex2(db);
  Stat o;
  o.m = m;
  o.s = a.s * fa + b.s * fb;
  o.t = ENT ? (a.t + da * a.s) * fa + (b.t + db * b.s) * fb : 0.f;
  return o;
}

// Adds logit x to the sums.
template <bool ENT>
__device__ __forceinline__ void stat_add(Stat& a, float x, float c) {
  if (x > a.m) {
    const float d = fmaxf((a.m - x) * c, kMinExp);
    const float f = ex2(d);
    if (ENT) a.t = (a.t + d * a.s) * f;
    a.s *= f;
    a.m = x;
  }
  // a maximum of -inf: every logit so far is -inf and weighs 0 (or is NaN)
  const float y = a.m == -INFINITY ? x : (x - a.m) * c;
  const float e = ex2(y);
  a.s += e;
  if (ENT) a.t = fmaf(e, y < kMinExp ? kMinExp : y, a.t);
}

template <bool ENT>
__device__ __forceinline__ Stat stat_block(Stat v, Stat* slots, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat w;
    w.m = __shfl_xor_sync(kAll, v.m, o);
    w.s = __shfl_xor_sync(kAll, v.s, o);
    w.t = ENT ? __shfl_xor_sync(kAll, v.t, o) : 0.f;
    v = stat_merge<ENT>(v, w, c);
  }
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  Stat o = slots[0];
  for (int w = 1; w < kLossWarps; ++w) o = stat_merge<ENT>(o, slots[w], c);
  __syncthreads();
  return o;
}

// A, Hc and the token's entry from the weights a, h of dlogp and dH.
__device__ __forceinline__ RowGrad row_grad(double a, double h, double logp, double H, double ln_s, float m, float s,
                                            float inv_t) {
  RowGrad g;
  g.m = m;
  g.a = g.h = g.at = 0.f;
  if (a == 0.0 && h == 0.0) return g;  // (NaN weights go on)
  const double k = -static_cast<double>(inv_t) / s;
  g.a = static_cast<float>(k * (a + (h != 0.0 ? h * (H - ln_s) : 0.0)));
  g.h = static_cast<float>(k * h * kLn2);
  double at = a * -expm1(logp);
  if (h != 0.0 && logp > -INFINITY) at -= h * exp(logp) * (logp + H);
  g.at = static_cast<float>(inv_t * at);
  return g;
}

// Everything a row gives besides its gradient's entries; run by one thread.
// kept_t: the token is in the kept set; x_t its logit.
template <Op OP, bool ENT>
__device__ __forceinline__ RowGrad row_scalars(const LossParams& p, RowStat* stats, int64_t row, Stat st, bool kept_t,
                                               float x_t) {
  RowGrad g;
  g.m = st.m;
  g.a = g.h = g.at = 0.f;
  const bool empty = st.s == 0.f;  // nothing kept, or only -inf
  const double log2_s = empty ? 0.0 : log2(static_cast<double>(st.s));
  double logp = -INFINITY;
  if (kept_t && !empty) logp = ((static_cast<double>(x_t) - st.m) * p.c - log2_s) * kLn2;
  const double H = ENT && !empty ? (log2_s - static_cast<double>(st.t) / st.s) * kLn2 : 0.0;
  const bool joins = logp != -INFINITY;  // (NaN joins)
  if (p.logp != nullptr) p.logp[row] = static_cast<float>(logp);
  if (ENT && p.entropy != nullptr) p.entropy[row] = static_cast<float>(H);
  if constexpr (OP == Op::kGrad) {
    const double a = joins && p.g_logp != nullptr ? p.g_logp[row] : 0.0;
    const double h = ENT && !empty ? p.g_entropy[row] : 0.0;
    g = row_grad(a, h, logp, H, log2_s * kLn2, st.m, st.s, p.inv_t);
  }
  if constexpr (OP == Op::kPolicy) {
    double loss = 0.0, kl = 0.0;
    if (joins) {
      const double adv = p.advantages[row];
      const double rho = p.old_logp != nullptr ? exp(logp - p.old_logp[row]) : 1.0;
      const double near = fmin(fmax(rho, p.clip_lo), p.clip_hi);
      loss = fmax(-adv * rho, -adv * near);
      if (rho != rho || logp != logp) loss = logp + rho;  // NaN goes through fmin and fmax unseen
      const bool bound = (adv > 0.0 && rho > p.clip_hi) || (adv < 0.0 && rho < p.clip_lo);
      double a = bound ? 0.0 : -adv * rho;
      if (p.ref_logp != nullptr) {
        const double q = p.ref_logp[row] - logp;
        const double eq = expm1(q);
        kl = eq - q;
        if (p.kl_coef != 0.0) {
          loss += p.kl_coef * kl;
          a -= p.kl_coef * eq;
        }
      }
      if (ENT) loss -= p.entropy_coef * H;
      if (p.grad != nullptr) {
        const double w = (p.weights != nullptr ? p.weights[row] : 1.0 / static_cast<double>(p.B)) *
                         (p.grad_loss != nullptr ? *p.grad_loss : 1.0);
        g = row_grad(w * a, ENT ? -p.entropy_coef * w : 0.0, logp, H, log2_s * kLn2, st.m, st.s, p.inv_t);
      }
    }
    p.row_loss[row] = static_cast<float>(loss);
    if (p.kl != nullptr) p.kl[row] = static_cast<float>(kl);
  }
  if constexpr (OP == Op::kPrefStats) {
    RowStat o;
    o.logp = logp;
    o.m = st.m;
    o.s = joins ? st.s : -1.f;
    stats[row] = o;
  }
  return g;
}

// Outputs of an ignored row, besides its gradient of 0.
template <Op OP>
__device__ __forceinline__ void row_ignored(const LossParams& p, RowStat* stats, int64_t row) {
  if (p.logp != nullptr) p.logp[row] = 0.f;
  if (p.entropy != nullptr) p.entropy[row] = 0.f;
  if constexpr (OP == Op::kPolicy) {
    p.row_loss[row] = 0.f;
    if (p.kl != nullptr) p.kl[row] = 0.f;
  }
  if constexpr (OP == Op::kPrefStats) {
    RowStat o;
    o.logp = 0.0;
    o.m = 0.f;
    o.s = -1.f;
    stats[row] = o;
  }
}

// Writes a row's gradient; token < 0: it has none of its own entry.
template <int DT, bool ENT>
__device__ __forceinline__ void write_grad(const LossParams& p, const void* xrow, const uint8_t* mrow, void* grow,
                                           RowGrad g, int64_t token) {
  const bool zero = g.a == 0.f && g.h == 0.f;
  for (int64_t j = threadIdx.x; j < p.V; j += kLossThreads) {
    float v = 0.f;
    if (j == token) {
      v = g.at;
    } else if (!zero && (mrow == nullptr || mrow[j] != 0)) {
      const float y = (load_logit<DT>(xrow, j) - g.m) * p.c;
      v = ex2(y) * (ENT ? fmaf(g.h, y < kMinExp ? kMinExp : y, g.a) : g.a);
    }
    store_grad<DT>(grow, j, v);
  }
}

// One CTA per row: the softmax sums in one pass, the row's values, and a
// second pass for the gradient.
template <int DT, Op OP, bool ENT>
__global__ void __launch_bounds__(kLossThreads) row_kernel(const LossParams p, RowStat* stats) {
  __shared__ Stat slots[kLossWarps];
  __shared__ RowGrad grad;
  const int64_t row = blockIdx.x;
  const void* xrow = row_at<DT>(p.logits, row, p.ld);
  const uint8_t* mrow = p.mask != nullptr ? p.mask + row * p.V : nullptr;
  const int64_t token = p.tokens[row];
  const bool ignored = token < 0 || token >= p.V;
  RowGrad g = {0.f, 0.f, 0.f, 0.f};
  if (ignored) {
    if (threadIdx.x == 0) row_ignored<OP>(p, stats, row);
  } else {
    Stat st = {-INFINITY, 0.f, 0.f};
    for (int64_t j = threadIdx.x; j < p.V; j += kLossThreads)
      if (mrow == nullptr || mrow[j] != 0) stat_add<ENT>(st, load_logit<DT>(xrow, j), p.c);
    st = stat_block<ENT>(st, slots, p.c);
    if (threadIdx.x == 0)
      grad = row_scalars<OP, ENT>(p, stats, row, st, mrow == nullptr || mrow[token] != 0, load_logit<DT>(xrow, token));
    __syncthreads();
    g = grad;
  }
  if (p.grad != nullptr)
    write_grad<DT, ENT>(p, xrow, mrow, row_at<DT>(p.grad, row, p.ld_grad), g,
                        ignored || (mrow != nullptr && mrow[token] == 0) ? -1 : token);
}

// out = sum of w[i] v[i] in one fixed order, in fp64 (w NULL: 1 / n).
__global__ void __launch_bounds__(1024) weighted_sum_kernel(const float* v, const float* w, int64_t n, float* out) {
  __shared__ double slots[32];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += static_cast<double>(v[i]) * (w != nullptr ? w[i] : 1.0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = slots[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (threadIdx.x == 0) *out = n == 0 ? 0.f : static_cast<float>(w != nullptr ? s : s / static_cast<double>(n));
  }
}

// Row [lo, hi) of sequence s, within [0, B] whatever starts holds.
__device__ __forceinline__ void sequence_rows(const int32_t* starts, int64_t s, int64_t B, int64_t& lo, int64_t& hi) {
  lo = min(max(static_cast<int64_t>(starts[s]), int64_t(0)), B);
  hi = min(max(static_cast<int64_t>(starts[s + 1]), lo), B);
}

// softplus(x) = log(1 + e^x) without overflow
__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }
__device__ __forceinline__ double sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

constexpr int kPairThreads = 128;

// One CTA per pair: the two sequences' sums in a fixed order, the pair's loss
// and the weight of dlogp of each sequence's rows.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const LossParams p, const PrefParams q,
                                                            const RowStat* stats, double* coef) {
  __shared__ double sum_slots[kPairThreads / 32];
  __shared__ int cnt_slots[kPairThreads / 32];
  const int64_t i = blockIdx.x;
  double seq[2], n[2];
  for (int k = 0; k < 2; ++k) {
    int64_t lo, hi;
    sequence_rows(q.starts, 2 * i + k, p.B, lo, hi);
    double s = 0.0;
    int cnt = 0;
    for (int64_t row = lo + threadIdx.x; row < hi; row += kPairThreads) {
      const RowStat st = stats[row];
      if (!(st.s < 0.f)) {
        s += st.logp;
        ++cnt;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(kAll, s, o);
      cnt += __shfl_xor_sync(kAll, cnt, o);
    }
    if ((threadIdx.x & 31) == 0) {
      sum_slots[threadIdx.x >> 5] = s;
      cnt_slots[threadIdx.x >> 5] = cnt;
    }
    __syncthreads();
    s = 0.0;
    cnt = 0;
    for (int w = 0; w < kPairThreads / 32; ++w) {
      s += sum_slots[w];
      cnt += cnt_slots[w];
    }
    __syncthreads();
    n[k] = q.length_norm && cnt > 0 ? 1.0 / cnt : 1.0;
    seq[k] = s * n[k];
  }
  if (threadIdx.x != 0) return;
  double rel[2];
  for (int k = 0; k < 2; ++k) {
    q.seq_logp[2 * i + k] = static_cast<float>(seq[k]);
    rel[k] = seq[k] - (q.ref != nullptr ? q.ref[2 * i + k] : 0.0);
  }
  const double ratio = rel[0] - rel[1];
  const double z = q.beta * ratio - q.margin;
  q.log_ratio[i] = static_cast<float>(ratio);
  q.pair_loss[i] = static_cast<float>((1.0 - q.smoothing) * softplus(-z) + (q.smoothing != 0.0 ? q.smoothing * softplus(z) : 0.0));
  const double w = (q.weights != nullptr ? q.weights[i] : 1.0 / static_cast<double>(q.P)) *
                   (p.grad_loss != nullptr ? *p.grad_loss : 1.0);
  const double d = w * q.beta * (q.smoothing * sigmoid(z) - (1.0 - q.smoothing) * sigmoid(-z));
  coef[2 * i] = d * n[0];
  coef[2 * i + 1] = -d * n[1];
}

// The last sequence that starts at or before row, -1 before the first.
__device__ __forceinline__ int64_t sequence_of(const int32_t* starts, int64_t n_starts, int64_t row) {
  int64_t lo = 0, hi = n_starts;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (starts[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

template <int DT>
__global__ void __launch_bounds__(kLossThreads) pref_grad_kernel(const LossParams p, const PrefParams q,
                                                                 const RowStat* stats, const double* coef) {
  const int64_t row = blockIdx.x;
  const void* xrow = row_at<DT>(p.logits, row, p.ld);
  const int64_t s = q.P > 0 ? sequence_of(q.starts, 2 * q.P + 1, row) : -1;
  RowGrad g = {0.f, 0.f, 0.f, 0.f};
  int64_t token = -1;
  if (s >= 0 && s < 2 * q.P) {
    const RowStat st = stats[row];
    if (!(st.s < 0.f)) {
      token = p.tokens[row];
      g = row_grad(coef[s], 0.0, st.logp, 0.0, 0.0, st.m, st.s, p.inv_t);
    }
  }
  write_grad<DT, false>(p, xrow, nullptr, row_at<DT>(p.grad, row, p.ld_grad), g, token);
}

// out_logp of rows that no sequence owns is 0.
__global__ void __launch_bounds__(kLossThreads) outside_kernel(const PrefParams q, int64_t B, float* logp) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kLossThreads + threadIdx.x;
  if (row >= B) return;
  const int64_t s = q.P > 0 ? sequence_of(q.starts, 2 * q.P + 1, row) : -1;
  if (s < 0 || s >= 2 * q.P) logp[row] = 0.f;
}

template <Op OP, bool ENT>
cudaError_t launch_rows(const LossParams& p, int dtype, RowStat* stats, cudaStream_t st) {
  const unsigned g = static_cast<unsigned>(p.B);
  if (dtype == QRITA_DTYPE_F32)
    row_kernel<QRITA_DTYPE_F32, OP, ENT><<<g, kLossThreads, 0, st>>>(p, stats);
  else
    row_kernel<QRITA_DTYPE_BF16, OP, ENT><<<g, kLossThreads, 0, st>>>(p, stats);
  return cudaGetLastError();
}

}  // namespace

int launch_logprobs(const LossParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return static_cast<int>(p.entropy != nullptr ? launch_rows<Op::kLogprobs, true>(p, dtype, nullptr, st)
                                               : launch_rows<Op::kLogprobs, false>(p, dtype, nullptr, st));
}

int launch_logprobs_grad(const LossParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return static_cast<int>(p.g_entropy != nullptr ? launch_rows<Op::kGrad, true>(p, dtype, nullptr, st)
                                                 : launch_rows<Op::kGrad, false>(p, dtype, nullptr, st));
}

int launch_policy(const LossParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.B > 0) {
    const bool ent = p.entropy != nullptr || p.entropy_coef != 0.0;
    const cudaError_t e = ent ? launch_rows<Op::kPolicy, true>(p, dtype, nullptr, st)
                              : launch_rows<Op::kPolicy, false>(p, dtype, nullptr, st);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  weighted_sum_kernel<<<1, 1024, 0, st>>>(p.row_loss, p.weights, p.B, p.loss);
  return static_cast<int>(cudaGetLastError());
}

// Workspace: RowStat[B], then double[2 P].
size_t pref_workspace_bytes(int64_t B, int64_t P) {
  const size_t n = static_cast<size_t>(B) * sizeof(RowStat) + static_cast<size_t>(P) * 2 * sizeof(double);
  return n < 256 ? 256 : (n + 255) / 256 * 256;
}

int launch_preference(const LossParams& p, const PrefParams& q, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  RowStat* stats = static_cast<RowStat*>(q.workspace);
  double* coef = reinterpret_cast<double*>(stats + p.B);
  cudaError_t e = cudaSuccess;
  if (p.B > 0) {
    e = launch_rows<Op::kPrefStats, false>([&] { LossParams f = p; f.grad = nullptr; return f; }(), dtype, stats, st);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (p.logp != nullptr) {
      outside_kernel<<<static_cast<unsigned>((p.B + kLossThreads - 1) / kLossThreads), kLossThreads, 0, st>>>(q, p.B, p.logp);
      if ((e = cudaGetLastError()) != cudaSuccess) return static_cast<int>(e);
    }
  }
  if (q.P > 0) {
    pair_kernel<<<static_cast<unsigned>(q.P), kPairThreads, 0, st>>>(p, q, stats, coef);
    if ((e = cudaGetLastError()) != cudaSuccess) return static_cast<int>(e);
  }
  weighted_sum_kernel<<<1, 1024, 0, st>>>(q.pair_loss, q.weights, q.P, p.loss);
  if ((e = cudaGetLastError()) != cudaSuccess) return static_cast<int>(e);
  if (p.B > 0 && p.grad != nullptr) {
    const unsigned g = static_cast<unsigned>(p.B);
    if (dtype == QRITA_DTYPE_F32) pref_grad_kernel<QRITA_DTYPE_F32><<<g, kLossThreads, 0, st>>>(p, q, stats, coef);
    else pref_grad_kernel<QRITA_DTYPE_BF16><<<g, kLossThreads, 0, st>>>(p, q, stats, coef);
    e = cudaGetLastError();
  }
  return static_cast<int>(e);
}

}  // namespace qrita
