// Losses over rows of logits and their gradients: log-probabilities of given
// tokens, the clipped policy loss with a KL term, and the preference loss on
// paired sequences.
//
// Qrita technical summary (gist.science, paper 2602.01518), "Problem
// statement": the candidate set and the drawn token feed reinforcement
// learning; these kernels score the drawn tokens under the same logits (and
// the same keep-mask).
//
// Everything is in base 2. With c = log2(e) * inv_temperature and m a kept logit
// within an octave of weight (1 / c) of the largest, a kept logit weighs
// e_j = 2^y_j, y_j = (x_j - m) c, and
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

#include "qrita_rows.cuh"

namespace qrita {
namespace {

// What row_kernel computes for a row.
enum Op : int { kOpLogprobs, kOpGrad, kOpPolicy, kOpPrefStats };

// g_j = 2^y_j (a + h y_j), y_j = (x_j - m) c; the token's own entry is `at`.
struct alignas(16) RowGrad {
  float m, a, h, at;
};

// Per-row record of the preference loss between its kernels.
struct RowStat {
  double logp;
  float m;
  float s;  // below 0: the row joins nothing
};

// What one thread reads of a row besides its logits, before any of the row's
// gradient is written (which may lie over the logits).
struct RowIn {
  float x_t;
  bool kept_t;
  float old_logp, ref_logp, adv;
  float w;          // weight in the gradient: weights[row] * grad_loss
  float g_logp, g_entropy;
};

// a > b for pairs in normal form (infinities included).
template <typename A, typename B>
__device__ __forceinline__ bool pair_above(A a, B b) { return a.hi != b.hi ? a.hi > b.hi : a.lo > b.lo; }

// v e^d where e^d alone may leave fp32 (d above kFarExp): by two factors of
// e^(d/2), which reach every product that fp32 holds of a normal v. 0 stays 0.
constexpr float kFarExp = 80.f;
__device__ __forceinline__ float times_far_exp(float v, F2 d) {
  if (v == 0.f && d.hi < INFINITY) return 0.f;
  const float h = expf(0.5f * d.hi) * (1.f + 0.5f * d.lo);
  return v * h * h;
}

// e^d - 1 of a pair. (Below -kFarExp, as an infinity's, d's low part is nothing.)
__device__ __forceinline__ float expm1_pair(F2 d) {
  const float more = expm1f(d.hi);
  return fabsf(d.hi) <= kFarExp ? fmaf(d.lo, more + 1.f, more) : more;
}

// e^q - 1 - q: its power series where the difference would lose digits (12
// terms leave less than 2^-26 of it for |q| <= 1).
__device__ __forceinline__ float exp_minus_tangent(F2 d) {
  const float q = d.hi;
  if (q > kFarExp) return times_far_exp(1.f, d);  // (1 + q is nothing beside it)
  if (fabsf(q) > 1.f) return expm1_pair(d) - q;
  float r = 1.f;
#pragma unroll
  for (int n = 13; n >= 3; --n) r = fmaf(r, q * (1.f / static_cast<float>(n)), 1.f);
  return fmaf(0.5f * q * q, r, d.lo * q);  // (q for its slope e^q - 1: d.lo q^2 is nothing)
}

// A, Hc and the token's entry from the weights a, h of dlogp and dH.
__device__ __forceinline__ RowGrad row_grad(float a, float h, float logp, float H, float ln_s, float m, float s,
                                            float inv_t) {
  RowGrad g;
  g.m = m;
  g.a = g.h = g.at = 0.f;
  if (a == 0.f && h == 0.f) return g;  // (NaN weights go on)
  const float k = -inv_t / s;
  g.a = k * (a + (h != 0.f ? h * (H - ln_s) : 0.f));
  g.h = k * (h * static_cast<float>(kLn2));
  float at = a * -expm1f(logp);
  if (h != 0.f && logp > -INFINITY) at -= h * expf(logp) * (logp + H);
  g.at = inv_t * at;
  return g;
}

template <int DT>
__device__ __forceinline__ RowIn row_in(const LossParams& p, int op, int64_t row, int64_t token) {
  RowIn in;
  in.x_t = Elem<DT>::load(static_cast<const unsigned char*>(p.logits) + row * p.ld * Elem<DT>::kBytes, token);
  in.kept_t = p.mask == nullptr || p.mask[row * p.V + token] != 0;
  in.old_logp = in.ref_logp = in.adv = in.g_logp = in.g_entropy = 0.f;
  in.w = 0.f;
  if (op == kOpGrad) {
    if (p.g_logp != nullptr) in.g_logp = p.g_logp[row];
    if (p.g_entropy != nullptr) in.g_entropy = p.g_entropy[row];
  } else if (op == kOpPolicy) {
    if (p.old_logp != nullptr) in.old_logp = p.old_logp[row];
    if (p.ref_logp != nullptr) in.ref_logp = p.ref_logp[row];
    in.adv = p.advantages[row];
    in.w = p.weights != nullptr ? p.weights[row] : p.inv_b;
    if (p.grad_loss != nullptr) in.w *= *p.grad_loss;
  }
  return in;
}

// A row's values on the way from its sums to its outputs.
struct RowVals {
  F2 logp;
  float lp, H;      // as they are given out
  float ln_s;
  F2 step;                  // -advantage * rho
  F2 q;                     // reference less logp
  bool joins, over, bound;  // over, bound: rho above the clip; the clip binds
};

// logp as a pair, so that ratios and their clip are decided on more than fp32
// has of a logp near -20. (fp64 would take this one thread longer than the
// row's whole pass: a function is hundreds of dependent instructions on a
// narrow pipe.)
template <bool ENT>
__device__ __forceinline__ RowVals row_vals(const LossParams& p, const RowIn& in, const Stat& st) {
  RowVals v;
  const bool empty = st.s.hi == 0.f;  // nothing kept, or only -inf
  const F2 S = sum_of(st);
  const F2 ln_s = empty ? f2_make(0.f, 0.f) : ln_pair(S);
  v.ln_s = ln_s.hi;
  // the mean of y_j ln2 under p
  const F2 mean = ENT && !empty ? mean_exponent(S, st.t) : f2_make(0.f, 0.f);
  // (a token that is not kept has probability 0 unless the row's sums are NaN)
  v.logp = f2_make(st.s.hi == st.s.hi ? -INFINITY : st.s.hi, 0.f);
  if (in.kept_t && !empty) {
    v.logp = logp_of(in.x_t, st.m, ln_s, p.inv_t, p.inv_t_lo);
  }
  v.lp = f2_float(v.logp);
  v.H = ENT && !empty ? f2_float(f2_sub(ln_s, mean)) : 0.f;
  v.joins = v.lp != -INFINITY;  // (NaN joins)
  v.step = v.q = f2_make(0.f, 0.f);
  v.over = v.bound = false;
  return v;
}

// The weights of a row's gradient.
template <bool ENT>
__device__ __forceinline__ RowGrad row_weights(const LossParams& p, int op, const RowIn& in, const Stat& st, RowVals& v) {
  float a = 0.f, h = 0.f;
  if (op == kOpGrad) {
    if (v.joins) a = in.g_logp;
    if (ENT && st.s.hi != 0.f) h = in.g_entropy;
  } else if (op == kOpPolicy && v.joins) {
    F2 d = f2_make(0.f, 0.f);  // ln rho
    if (p.old_logp != nullptr)
      d = isinf(in.old_logp) ? f2_make(-in.old_logp, 0.f) : f2_sub(v.logp, f2_make(in.old_logp, 0.f));
    // rho = 1 + (e^d - 1): near 1 one rounding of the product is what it costs
    const float adv_w = in.adv * in.w;
    if (d.hi > kFarExp) {
      v.step.hi = times_far_exp(-in.adv, d);
      a = times_far_exp(-adv_w, d);
    } else {
      const float more = expm1_pair(d);
      if (more > -0.5f) {
        v.step = f2_prod(-in.adv, more);
        f2_add(v.step, -in.adv);
        a = fmaf(-adv_w, more, -adv_w);
      } else {
        const float rho = expf(d.hi) * (1.f + d.lo);
        v.step.hi = -in.adv * rho;
        a = -adv_w * rho;
      }
    }
    // rho against the clip, on the logarithms
    v.over = pair_above(d, p.ln_hi);
    v.bound = (in.adv > 0.f && v.over) || (in.adv < 0.f && pair_above(p.ln_lo, d));
    if (v.bound) a = 0.f;
    if (p.ref_logp != nullptr) {
      v.q = isinf(in.ref_logp) ? f2_make(in.ref_logp, 0.f) : f2_sub(f2_make(in.ref_logp, 0.f), v.logp);
      const float kl_w = p.kl_coef * in.w;
      if (p.kl_coef != 0.f) a = v.q.hi > kFarExp ? a - times_far_exp(kl_w, v.q) : fmaf(-kl_w, expm1_pair(v.q), a);
    }
    if (v.lp != v.lp) a = v.lp;
    if (ENT) h = -p.entropy_coef * in.w;
  }
  return row_grad(a, h, v.lp, v.H, v.ln_s, st.m, st.s.hi, p.inv_t);
}

// Writes a row's values (after row_weights where the operator has them).
template <bool ENT>
__device__ __forceinline__ void row_out(const LossParams& p, int op, RowStat* stats, int64_t row, const RowIn& in,
                                        const Stat& st, const RowVals& v) {
  if (p.logp != nullptr) p.logp[row] = v.lp;
  if (ENT && p.entropy != nullptr) p.entropy[row] = v.H;
  if (op == kOpPolicy) {
    float loss = 0.f, kl = 0.f;
    if (v.joins) {
      const LossPair clip = v.over ? p.clip_hi : p.clip_lo;
      F2 term = v.bound ? f2_mul(f2_make(clip.hi, clip.lo), -in.adv) : v.step;  // rounded once, with its terms
      if (isinf(term.hi)) term.lo = 0.f;
      if (p.ref_logp != nullptr) {
        kl = exp_minus_tangent(v.q);
        if (p.kl_coef != 0.f) term.lo += v.q.hi > kFarExp ? times_far_exp(p.kl_coef, v.q) : p.kl_coef * kl;
      }
      if (ENT) term.lo = fmaf(-p.entropy_coef, v.H, term.lo);
      loss = v.lp != v.lp ? v.lp : f2_float(term);
    }
    p.row_loss[row] = loss;
    if (p.kl != nullptr) p.kl[row] = kl;
  } else if (op == kOpPrefStats) {
    RowStat o;
    o.logp = static_cast<double>(v.logp.hi) + v.logp.lo;
    o.m = st.m;
    o.s = v.joins ? st.s.hi : -1.f;
    stats[row] = o;
  }
}

// Outputs of an ignored row, besides its gradient of 0.
__device__ __forceinline__ void row_ignored(const LossParams& p, int op, RowStat* stats, int64_t row) {
  if (p.logp != nullptr) p.logp[row] = 0.f;
  if (p.entropy != nullptr) p.entropy[row] = 0.f;
  if (op == kOpPolicy) {
    p.row_loss[row] = 0.f;
    if (p.kl != nullptr) p.kl[row] = 0.f;
  }
  if (op == kOpPrefStats) {
    RowStat o;
    o.logp = 0.0;
    o.m = 0.f;
    o.s = -1.f;
    stats[row] = o;
  }
}

template <bool ENT>
__device__ __forceinline__ float grad_one(float x, const RowGrad& g, float c) {
  const float y = (x - g.m) * c;
  return ex2(y) * (ENT ? fmaf(g.h, y < kMinExp ? kMinExp : y, g.a) : g.a);
}

// The entries of a row whose gradient is that of several log-probabilities
// (qrita_token_scores_grad): K given ids with an incoming gradient g_i each. With a
// the sum of g_i over the ids of probability above 0, a logit's own entry is
//   inv_t (G_j - p_j (a + h (log p_j + H))),  G_j the sum of g_i over i with id j,
// taken as G_j (1 - p_j) - p_j (a - G_j + ...), 1 - p_j by expm1. A thread keeps the
// logits of its ids (read before a gradient is written over them), on their way while
// the row is summed; ids and gradients are read again where they are used, and wait
// for the last step in the sums' shared memory. Sums of g_i are fp64 over a row and
// pairs of fp32 over an id that is listed more than once, each in one order: a - G_j is
// what is left of their difference. (An id's places are counted first, two instructions
// an id: with its sum taken on the way 256 ids of 512 x 151936 87 us in fp32, and 64 ids
// of 255 x 50021 34 in fp64.)
// (512 x 151936 bf16: one id a row 56 us, 20 59, 64 61, 256 85, half of them one id 94;
// 255 x 50021 fp32 with entropies: 64 ids 23 us, 256 33.)
struct ManyRow {
  F2 a, ln_s;
  float m, H, h;
};

template <int THREADS>
struct Many {
  static constexpr int kEach = kMaxGradIds / THREADS;
  float x[kEach];  // -inf: its probability is 0, or there is no such id

  // Whether any incoming gradient of the row is not 0 (by the whole block).
  // `logit` gives the logit of an id in this CTA's share (-inf of one that is not
  // kept, or lies in another CTA's).
  template <typename F>
  __device__ __forceinline__ bool load(const LossParams& p, int64_t row, F logit) {
    bool any = threadIdx.x == 0 && p.g_entropy != nullptr && p.g_entropy[row] != 0.f;
    int id[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = threadIdx.x + i * THREADS;
      id[i] = -1;
      x[i] = -INFINITY;
      if (k < p.K && p.g_logp != nullptr) {
        const float g = p.g_logp[row * p.K + k];
        id[i] = p.tokens[row * p.K + k];
        if (id[i] >= p.V) id[i] = -1;
        any = any || (id[i] >= 0 && g != 0.f);
      }
    }
    any = __syncthreads_or(any);
    if (any) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (id[i] >= 0) x[i] = logit(i, static_cast<int64_t>(id[i]));
    }
    return any;
  }

  // The warps' sums of the gradients of this CTA's ids that have a probability.
  __device__ __forceinline__ void add_up(const LossParams& p, int64_t row, double* sums) const {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (x[i] != -INFINITY) sum += p.g_logp[row * p.K + threadIdx.x + i * THREADS];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  }

  // The CTA's own to every CTA of the cluster, before its barrier, by one warp and
  // after one of the block; every warp's sum is there.
  __device__ __forceinline__ static void send(const double* sums, uint32_t rank, uint32_t C, double* ranks) {
    double a = 0.0;
    for (int i = 0; i < THREADS / 32; ++i) a += sums[i];
    const uint32_t lane = threadIdx.x & 31;
    if (lane < C) {
      const uint32_t at = map_rank(smem_u32(&ranks[rank]), lane);
      st_dsmem_u32(at, static_cast<uint32_t>(__double2loint(a)));
      st_dsmem_u32(at + 4, static_cast<uint32_t>(__double2hiint(a)));
    }
  }

  // Ids and gradients to shared memory that the sums have left.
  __device__ __forceinline__ static void keep(const LossParams& p, int64_t row, StatSlots<THREADS>& slots) {
    static_assert(4 * THREADS >= 2 * kMaxGradIds, "ids and gradients fit in the sums' place");
    int* ids = reinterpret_cast<int*>(slots.m);
    float* g = reinterpret_cast<float*>(ids + kMaxGradIds);
    if (p.g_logp == nullptr) return;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = threadIdx.x + i * THREADS;
      if (k >= kMaxGradIds) break;
      ids[k] = k < p.K ? p.tokens[row * p.K + k] : -1;
      g[k] = k < p.K ? p.g_logp[row * p.K + k] : 0.f;
    }
  }

  // One thread's: the row's gradient weights from its sums.
  template <bool ENT>
  __device__ __forceinline__ static RowGrad weights(const LossParams& p, int64_t row, const Stat& st, const RowVals& v,
                                                    const double* ranks, ManyRow& r) {
    double a = 0.0;
    for (uint32_t i = 0; i < p.C; ++i) a += ranks[i];
    if (st.s.hi != st.s.hi) a = st.s.hi;  // (NaN for the whole row)
    r.a.hi = static_cast<float>(a);
    r.a.lo = static_cast<float>(a - r.a.hi);
    r.h = ENT && st.s.hi != 0.f ? p.g_entropy[row] : 0.f;
    r.H = v.H;
    r.m = st.m;
    r.ln_s = st.s.hi != 0.f ? ln_pair(sum_of(st)) : f2_make(0.f, 0.f);
    return row_grad(r.a.hi, r.h, -INFINITY, v.H, v.ln_s, st.m, st.s.hi, p.inv_t);
  }

  // The entries of this CTA's ids, over what a barrier before this has seen written.
  template <int DT>
  __device__ __forceinline__ void write(const LossParams& p, const ManyRow& r, const StatSlots<THREADS>& slots,
                                        unsigned char* grow) const {
    const int* ids = reinterpret_cast<const int*>(slots.m);
    const float* g = reinterpret_cast<const float*>(ids + kMaxGradIds);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = threadIdx.x + i * THREADS;
      if (x[i] == -INFINITY) continue;
      const int id = ids[k];
      int places = 0;
      for (int j = 0; j < p.K; j += 4) {  // (behind the last id are ids of -1)
        const int4 v = *reinterpret_cast<const int4*>(ids + j);
        places += v.x == id;
        places += v.y == id;
        places += v.z == id;
        places += v.w == id;
      }
      F2 sum = f2_make(g[k], 0.f);
      if (places > 1) {  // the first of them writes
        bool first = true;
        for (int j = 0; j < k && first; ++j) first = ids[j] != id;
        if (!first) continue;
        for (int j = k + 1; j < p.K; ++j)
          if (ids[j] == id) f2_add(sum, g[j]);
      }
      const float lp = f2_float(logp_of(x[i], r.m, r.ln_s, p.inv_t, p.inv_t_lo)), prob = expf(lp);
      const float G = f2_float(sum);
      float rest = isfinite(r.a.hi) ? f2_float(f2_sub(r.a, sum)) : r.a.hi - G;
      // (a probability of 0 takes nothing of it, not 0 * inf where log p, or h times it, has left fp32)
      if (r.h != 0.f && prob != 0.f) rest = fmaf(r.h, lp + r.H, rest);
      Elem<DT>::store(grow, id, p.inv_t * (G * -expm1f(lp) - prob * rest));
    }
  }
};

// Writes this CTA's share of a row's gradient. token < 0: no entry of its
// own. Every unit is read and then written by the same thread, so the
// gradient may lie over the logits.
template <int THREADS, int DT, bool ENT>
__device__ __forceinline__ void write_grad(const LossParams& p, const Share<DT>& sh, int64_t row, const RowGrad& g,
                                           int64_t token) {
  using E = Elem<DT>;
  constexpr int N = E::kUnit / 2;
  unsigned char* grow = static_cast<unsigned char*>(p.grad) + row * p.ld_grad * E::kBytes;
  unsigned char* gu = grow + sh.head * E::kBytes;
  const bool vec = (reinterpret_cast<uintptr_t>(gu) & 15u) == 0;
  const bool zero = g.a == 0.f && g.h == 0.f;
  const float2 nm = both(-g.m), cc = both(p.c.hi), aa = both(g.a), hh = both(g.h);
  auto put = [&](int64_t u, const float2 (&v)[N]) {
    if (vec) {
      __stcs(reinterpret_cast<uint4*>(gu + u * 16), E::pack(v));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        E::store(gu, u * E::kUnit + 2 * i, v[i].x);
        E::store(gu, u * E::kUnit + 2 * i + 1, v[i].y);
      }
    }
  };
  if (zero) {
    float2 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = both(0.f);
    for (int64_t u = sh.u_lo + threadIdx.x; u < sh.u_hi; u += THREADS) put(u, v);
  } else {
    for (int64_t u0 = sh.u_lo + threadIdx.x; u0 < sh.u_hi; u0 += THREADS * kUnroll) {
      uint4 w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (u0 + k * THREADS < sh.u_hi) w[k] = __ldcs(static_cast<const uint4*>(sh.unit(u0 + k * THREADS)));
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t u = u0 + k * THREADS;
        if (u >= sh.u_hi) break;
        float2 x[N], v[N];
        E::unpack(w[k], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 y = mul2(add2(x[i], nm), cc);
          const float2 e = make_float2(ex2(y.x), ex2(y.y));
          v[i] = ENT ? mul2(e, fma2(hh, make_float2(y.x < kMinExp ? kMinExp : y.x, y.y < kMinExp ? kMinExp : y.y), aa))
                     : mul2(e, aa);
        }
        put(u, v);
      }
    }
  }
  if (sh.ends && threadIdx.x < Share<DT>::kEnds) {
    const int64_t j = sh.end_index(threadIdx.x);
    if (j >= 0) {
      float v = 0.f;
      if (!zero) v = grad_one<ENT>(E::load(sh.x, j), g, p.c.hi);
      E::store(grow, j, v);
    }
  }
  // the token's own entry, by the CTA that wrote its place
  if (token >= 0 && sh.owns(token)) {
    __syncthreads();
    if (threadIdx.x == 0) E::store(grow, token, g.at);
  }
}

// Blocks of row_kernel on an SM: five where 48 registers a thread are enough
// (log-probabilities of 1500 x 262144 bf16 113 us, with four 124; of 700 x 32000 8.4
// and 9.9; of 1024 x 262144, whose last wave is fuller with four, 91 and 85).
template <int DT, bool ENT>
constexpr int kRowBlocks = DT == QRITA_DTYPE_BF16 && !ENT ? 5 : kLossBlocks;

// A cluster of C CTAs per row, in one pass over HBM for the sums: each CTA
// streams its share of the row, the shares merge through distributed shared
// memory, and rank 0 writes the row's values. A gradient (here only of rows too
// long for resident_kernel) takes a second pass over the share. HBM bounds it:
// log-probabilities of 1500 x 262144 bf16 113 us (7.0 TB/s), of 1024 rows 91 us
// (5.9 TB/s: 1.3 waves of blocks); with entropies 1024 rows 89 us (1.7 waves).
template <int THREADS, int DT, bool ENT, bool MANY = false>
__global__ void __launch_bounds__(THREADS, kLossThreads * kRowBlocks<DT, ENT> / THREADS)
row_kernel(const LossParams p, RowStat* stats, int op) {
  using E = Elem<DT>;
  constexpr int N = E::kUnit / 2;
  __shared__ StatSlots<THREADS> slots;
  __shared__ RowGrad grad;
  __shared__ RowIn in;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t C = p.C;
  const int64_t row = cluster_id();
  const int64_t token = MANY ? -1 : p.tokens[row];
  const uint32_t rank = C > 1 ? cluster_rank() : 0u;
  const Share<DT> sh(p, row, rank);
  RowGrad g = {0.f, 0.f, 0.f, 0.f};
  Many<THREADS> many;
  __shared__ double many_sums[MANY ? THREADS / 32 : 1], many_ranks[MANY ? kMaxRanks : 1];
  __shared__ ManyRow many_row;
  bool ignored = false;
  if constexpr (MANY)
    ignored = !many.load(p, row, [&](int, int64_t id) { return sh.owns(id) ? E::load(sh.x, id) : -INFINITY; });
  else
    ignored = token < 0 || token >= p.V;
  if (ignored) {  // (the same in every CTA of the cluster)
    if (!MANY && threadIdx.x == 0 && rank == 0) row_ignored(p, op, stats, row);
    if (p.grad != nullptr) write_grad<THREADS, DT, ENT>(p, sh, row, g, -1);
    return;
  }
  if (C > 1) cluster_arrive_relaxed();  // every CTA of the cluster runs before its memory is written
  if (!MANY && threadIdx.x == 32) in = row_in<DT>(p, op, row, token);  // (read after the sums' barrier)
  Running<ENT> run;
  int64_t u0 = sh.u_lo + threadIdx.x;
  // whole steps of the block first: no unit of theirs needs a check
  for (int64_t full = sh.u_lo + (sh.u_hi - sh.u_lo) / (THREADS * kUnroll) * (THREADS * kUnroll); u0 < full;
       u0 += THREADS * kUnroll) {
    uint4 w[kUnroll];
    float2 x[kUnroll * N];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) w[k] = load_unit(sh.unit(u0 + k * THREADS));
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) E::unpack(w[k], reinterpret_cast<float2(&)[N]>(x[k * N]));
    run.add_unit(x, p.c);
  }
  for (; u0 < sh.u_hi; u0 += THREADS) {
    float2 x[N];
    E::unpack(load_unit(sh.unit(u0)), x);
    run.add_unit(x, p.c);
  }
  if (sh.ends && threadIdx.x < Share<DT>::kEnds) {
    const int64_t j = sh.end_index(threadIdx.x);
    if (j >= 0) run.add_one(E::load(sh.x, j), p.c);
  }
  if constexpr (MANY) many.add_up(p, row, many_sums);
  const Stat st = row_stat(run, p.c, rank, C, slots, [&]() {
    if constexpr (MANY) Many<THREADS>::send(many_sums, rank, C, many_ranks);
  });
  RowVals v;
  if (threadIdx.x == 0 && (rank == 0 || p.grad != nullptr)) {
    if constexpr (MANY) {
      v = row_vals<ENT>(p, RowIn{}, st);
      grad = Many<THREADS>::template weights<ENT>(p, row, st, v, many_ranks, many_row);
    } else {
      v = row_vals<ENT>(p, in, st);
      if (p.grad != nullptr || op == kOpPolicy) grad = row_weights<ENT>(p, op, in, st, v);
    }
    if (p.grad == nullptr) row_out<ENT>(p, op, stats, row, in, st, v);
  }
  if (p.grad == nullptr) return;
  __syncthreads();
  if (!MANY && threadIdx.x == 0 && rank == 0) row_out<ENT>(p, op, stats, row, in, st, v);
  if constexpr (MANY) many.keep(p, row, slots);
  g = grad;
  write_grad<THREADS, DT, ENT>(p, sh, row, g, token);
  if constexpr (MANY) {
    __syncthreads();
    many.template write<DT>(p, many_row, slots, static_cast<unsigned char*>(p.grad) + row * p.ld_grad * E::kBytes);
  }
}

// ---------------------------------------------------------------------------
// The same over a kept set. The mask is read once, 16 ids to a load: its bits go
// to a map in shared memory, the kept ids to a list. Where the list holds them
// (top-k sets, most top-p sets), all their logits are then loaded at once (a load
// for each as it is found would put one memory latency after another), and the
// gradient is a row of zeros, stored while the sums are taken, with the listed
// entries put over them. The list's order is that of the atomics on its length:
// its sums are taken in 64-bit fixed point, which no order changes. Rows that
// keep more are walked by the map, 16 bytes of logits at a time and only where a
// bit is set, once for the sums and once for the gradient.
//
// Log-probabilities over 64 kept ids of 1024 x 262144 bf16: 53 us, the mask at
// 5.0 TB/s (78 us when a unit of mask bytes led to its logits at once); half of
// all ids kept, 148 us for 805 MB. Policy loss over the kept sets of a mixed top-k
// and top-p batch of that size (a fifth of the rows keep 16 thousand ids or more)
// 188 us; with a list of half the length and no map (rows beyond it read the mask
// again before each load, and again for the gradient) 373. 128 x 151936 fp32 with
// 64 kept: 22 us for 97 MB of mask and zeros; scan, merge and stores of one wave
// of blocks follow one another. Four mask units in flight instead of eight cost
// 4 %; a list in id order by prefix sums over the map, two barriers more, 12 % of
// the log-probabilities of 64 x 128256.
// ---------------------------------------------------------------------------
constexpr int kKeptUnit = 16;
constexpr int kMaskUnroll = 8;  // units of the mask, or kept logits, a thread has in flight
// Ids of a CTA's bit map, and the entries of its list.
template <int THREADS>
constexpr int kKeptMap = THREADS == kLossThreads ? 128 * 1024 : kShortRow;
template <int THREADS>
constexpr int kKeptList = 16 * THREADS;
// A listed logit weighs at most 1 and a CTA lists at most 2^12: sums stay
// below 2^63 at this scale, and a weight is rounded by 2^-48 of the largest.
constexpr float kKeptScale = 0x1p47f;

__device__ __forceinline__ F2 kept_pair(unsigned long long v) {
  const F2 a = f2_from_u64(v);
  return f2_make(a.hi * 0x1p-47f, a.lo * 0x1p-47f);
}

// Zeros to elements [lo, hi) of a row, by the whole block.
template <int THREADS, int DT>
__device__ __forceinline__ void zero_range(unsigned char* grow, int64_t lo, int64_t hi) {
  using E = Elem<DT>;
  const uintptr_t a = reinterpret_cast<uintptr_t>(grow + lo * E::kBytes), b = reinterpret_cast<uintptr_t>(grow + hi * E::kBytes);
  uintptr_t va = (a + 15u) & ~static_cast<uintptr_t>(15u), vb = b & ~static_cast<uintptr_t>(15u);
  if (va > vb) va = vb = b;  // no whole unit: all of it is the head
  for (uintptr_t q = va + 16u * threadIdx.x; q < vb; q += 16u * THREADS)
    *reinterpret_cast<uint4*>(q) = make_uint4(0u, 0u, 0u, 0u);
  const int64_t head = static_cast<int64_t>(va - a) / E::kBytes, tail = static_cast<int64_t>(b - vb) / E::kBytes;
  if (threadIdx.x < head) E::store(grow, lo + threadIdx.x, 0.f);
  if (threadIdx.x < tail) E::store(grow, hi - tail + threadIdx.x, 0.f);
}

template <int THREADS, int DT, bool ENT, bool MANY = false>
__global__ void __launch_bounds__(THREADS, kLossThreads * kLossBlocks / THREADS) kept_kernel(const LossParams p, int op) {
  using E = Elem<DT>;
  __shared__ StatSlots<THREADS> slots;
  __shared__ RowGrad grad;
  __shared__ RowIn in;
  __shared__ int count;  // kept ids, up to where the list overflows
  __shared__ unsigned long long sums[2];
  __shared__ int list[kKeptList<THREADS>];  // ids within the CTA's range
  // the kept bits of each unit; where there is a list, its logits take their place
  constexpr int kMapBytes = kKeptMap<THREADS> / 8, kLogitBytes = 4 * kKeptList<THREADS>;
  __shared__ uint4 shared_units[(kMapBytes > kLogitBytes ? kMapBytes : kLogitBytes) / 16];
  unsigned short* map = reinterpret_cast<unsigned short*>(shared_units);
  float* list_x = reinterpret_cast<float*>(shared_units);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const uint32_t C = p.C;
  const int64_t row = cluster_id();
  const uint32_t rank = C > 1 ? cluster_rank() : 0u;
  const int64_t token = MANY ? -1 : p.tokens[row];
  const int64_t V = p.V;
  const unsigned char* xrow = static_cast<const unsigned char*>(p.logits) + row * p.ld * E::kBytes;
  const uint8_t* mrow = p.mask + row * V;
  unsigned char* grow = p.grad != nullptr ? static_cast<unsigned char*>(p.grad) + row * p.ld_grad * E::kBytes : nullptr;
  // units of 16 ids on the mask's 16-byte boundaries; the ids before the first
  // unit are rank 0's, those behind the last one the last rank's
  const int64_t head = min(V, static_cast<int64_t>((16u - (reinterpret_cast<uintptr_t>(mrow) & 15u)) & 15u));
  const int64_t nu = static_cast<int64_t>(static_cast<uint64_t>(V - head) / kKeptUnit);
  const int64_t u_lo = min(nu, static_cast<int64_t>(rank) * p.per), u_hi = rank == C - 1 ? nu : min(nu, u_lo + p.per);
  const int64_t lo = rank == 0 ? 0 : head + u_lo * kKeptUnit, hi = rank == C - 1 ? V : head + u_hi * kKeptUnit;
  const int n_map = static_cast<int>(min(u_hi - u_lo, static_cast<int64_t>(INT32_MAX)));
  const bool mapped = n_map <= kKeptMap<THREADS> / kKeptUnit;
  const uint8_t* mu = mrow + head + u_lo * kKeptUnit;
  uint4 m_in[kMaskUnroll];
  auto fetch = [&](int u0) {
#pragma unroll
    for (int k = 0; k < kMaskUnroll; ++k)
      if (u0 + k * THREADS < n_map) m_in[k] = load_unit(mu + static_cast<int64_t>(u0 + k * THREADS) * kKeptUnit);
  };
  if (mapped) fetch(tid);  // (on its way while the token is)
  Many<THREADS> many;
  __shared__ double many_sums[MANY ? THREADS / 32 : 1], many_ranks[MANY ? kMaxRanks : 1];
  __shared__ ManyRow many_row;
  bool ignored = false;
  if constexpr (MANY)
    ignored = !many.load(p, row, [&](int, int64_t id) {
      return id >= lo && id < hi && mrow[id] != 0 ? E::load(xrow, id) : -INFINITY;
    });
  else
    ignored = token < 0 || token >= V;
  if (ignored) {  // (the same in every CTA of the cluster)
    if (!MANY && tid == 0 && rank == 0) row_ignored(p, op, nullptr, row);
    if (grow != nullptr) zero_range<THREADS, DT>(grow, lo, hi);
    return;
  }
  if (C > 1) cluster_arrive_relaxed();  // every CTA of the cluster runs before its memory is written
  if (tid == 0) {
    count = mapped ? 0 : INT32_MAX;
    sums[0] = sums[1] = 0ull;
  }
  if (!MANY && tid == 32) in = row_in<DT>(p, op, row, token);  // (read after the sums' barrier)
  int64_t end_j = -1;  // this thread's id before the first unit or behind the last
  if (rank == 0 && tid < head) end_j = tid;
  const int64_t tail = head + nu * kKeptUnit;
  if (rank == C - 1 && tid >= 32 && tail + tid - 32 < V) end_j = tail + tid - 32;
  const bool end_kept = end_j >= 0 && mrow[end_j] != 0;
  __syncthreads();
  if (mapped) {
    const int j0 = static_cast<int>(head + u_lo * kKeptUnit - lo);
    for (int u0 = tid; u0 < n_map; u0 += THREADS * kMaskUnroll) {
      if (u0 != tid) fetch(u0);
#pragma unroll
      for (int k = 0; k < kMaskUnroll; ++k) {
        const int u = u0 + k * THREADS;
        if (u >= n_map) break;
        uint32_t bits = kept_bits(m_in[k]);
        map[u] = static_cast<unsigned short>(bits);
        if (bits == 0u || *reinterpret_cast<volatile int*>(&count) > kKeptList<THREADS>) continue;
        int at = atomicAdd(&count, __popc(bits));
        for (; bits != 0u && at < kKeptList<THREADS>; ++at, bits &= bits - 1u) list[at] = j0 + u * kKeptUnit + __ffs(bits) - 1;
      }
    }
    if (end_kept) {
      const int at = atomicAdd(&count, 1);
      if (at < kKeptList<THREADS>) list[at] = static_cast<int>(end_j - lo);
    }
  }
  __syncthreads();
  const bool listed = count <= kKeptList<THREADS>;
  const bool over_logits = p.grad == p.logits;
  const bool vec = (reinterpret_cast<uintptr_t>(xrow + head * E::kBytes) & 15u) == 0;
  // Walked units: 16 bytes of logits, U of them. Their bits are in the map, or
  // (shares beyond the map's length, rows of millions) in U aligned mask bytes.
  constexpr int U = E::kUnit, N = U / 2;
  const int64_t e_lo = head + u_lo * kKeptUnit, n_u = (u_hi - u_lo) * (kKeptUnit / U);
  auto bits_of = [&](int64_t u) {
    if (mapped) {
      const unsigned char* at = reinterpret_cast<const unsigned char*>(map);
      return U == 8 ? static_cast<uint32_t>(at[u]) : at[u >> 1] >> (4 * (u & 1)) & 15u;
    }
    uint4 m = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(mrow + e_lo + u * U);
    m.x = w[0];
    if (U == 8) m.y = w[1];
    return kept_bits(m);
  };
  // the kept logits of unit u (anything where none is kept)
  auto load = [&](int64_t u, uint32_t bits) {
    const int64_t j = e_lo + u * U;
    if (bits == 0u) return make_uint4(0u, 0u, 0u, 0u);
    if (vec) return load_unit(xrow + j * E::kBytes);
    float2 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i].x = bits >> (2 * i) & 1u ? E::load(xrow, j + 2 * i) : 0.f;
      x[i].y = bits >> (2 * i + 1) & 1u ? E::load(xrow, j + 2 * i + 1) : 0.f;
    }
    return E::pack(x);
  };
  // -inf where they are not kept
  auto expand = [&](uint4 w, uint32_t bits, float2 (&x)[N]) {
    E::unpack(w, x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!(bits >> (2 * i) & 1u)) x[i].x = -INFINITY;
      if (!(bits >> (2 * i + 1) & 1u)) x[i].y = -INFINITY;
    }
  };
  if constexpr (MANY) many.add_up(p, row, many_sums);  // (barriers follow)
  Stat st;
  if (listed) {
    float m = -INFINITY;
    bool bad = false;  // NaN has no fixed point
    for (int i0 = tid; i0 < count; i0 += THREADS * kMaskUnroll) {
      float x[kMaskUnroll];
#pragma unroll
      for (int k = 0; k < kMaskUnroll; ++k)
        x[k] = i0 + k * THREADS < count ? E::load(xrow, lo + list[i0 + k * THREADS]) : -INFINITY;
#pragma unroll
      for (int k = 0; k < kMaskUnroll; ++k) {
        if (i0 + k * THREADS < count) list_x[i0 + k * THREADS] = x[k];
        m = fmaxf(m, x[k]);
        bad = bad || x[k] != x[k] || x[k] == INFINITY;
      }
    }
    if (grow != nullptr && !over_logits) zero_range<THREADS, DT>(grow, lo, hi);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if ((tid & 31) == 0) slots.m[tid >> 5] = m;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < THREADS / 32; ++w) m = fmaxf(m, slots.m[w]);
    unsigned long long s = 0ull, t = 0ull;
    for (int i = tid; i < count; i += THREADS) {
      const float x = list_x[i];
      const float y = x == -INFINITY ? kMinExp : fmaxf(scaled(x - m, p.c), kMinExp);
      const float e = bad ? 0.f : ex2(y);
      s += round_u64(e * kKeptScale);
      if (ENT) t += round_u64(e * -y * kKeptScale);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(kAll, s, o);
      if (ENT) t += __shfl_xor_sync(kAll, t, o);
    }
    if ((tid & 31) == 0) {
      atomicAdd(&sums[0], s);
      if (ENT) atomicAdd(&sums[1], t);
    }
    __syncthreads();
    st.m = m;
    st.s = bad ? f2_make(NAN, NAN) : kept_pair(sums[0]);
    st.t = bad ? f2_make(NAN, NAN) : kept_pair(sums[1]);
    st.t = f2_make(-st.t.hi, -st.t.lo);
  } else {
    Running<ENT> run;
    int64_t u = tid;
    for (; u + (kUnroll - 1) * THREADS < n_u; u += kUnroll * THREADS) {
      uint32_t bits[kUnroll];
      uint4 w[kUnroll];
      float2 x[kUnroll * N];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) bits[k] = bits_of(u + k * THREADS);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) w[k] = load(u + k * THREADS, bits[k]);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) expand(w[k], bits[k], reinterpret_cast<float2(&)[N]>(x[k * N]));
      run.add_unit(x, p.c);
    }
    for (; u < n_u; u += THREADS) {
      float2 x[N];
      const uint32_t bits = bits_of(u);
      expand(load(u, bits), bits, x);
      run.add_unit(x, p.c);
    }
    if (end_kept) run.add_one(E::load(xrow, end_j), p.c);
    put_stat(run, slots);
    __syncthreads();
    if (tid < 32) st = warp_stat<THREADS, ENT>(p.c, slots);
  }
  if (C > 1) cluster_wait();
  if constexpr (MANY) {
    if (tid < 32) Many<THREADS>::send(many_sums, rank, C, many_ranks);
  }
  cluster_stat<ENT>(st, p.c, rank, C, slots.ranks);
  RowVals v;
  if (tid == 0 && (rank == 0 || grow != nullptr)) {
    if constexpr (MANY) {
      v = row_vals<ENT>(p, RowIn{}, st);
      grad = Many<THREADS>::template weights<ENT>(p, row, st, v, many_ranks, many_row);
    } else {
      v = row_vals<ENT>(p, in, st);
      if (grow != nullptr || op == kOpPolicy) grad = row_weights<ENT>(p, op, in, st, v);
    }
    if (grow == nullptr) row_out<ENT>(p, op, nullptr, row, in, st, v);
  }
  if (grow == nullptr) return;
  __syncthreads();
  if (!MANY && tid == 0 && rank == 0) row_out<ENT>(p, op, nullptr, row, in, st, v);
  if constexpr (MANY) many.keep(p, row, slots);
  const RowGrad g = grad;
  const bool zero = g.a == 0.f && g.h == 0.f;
  if (listed) {
    if (over_logits) {  // (the other CTAs have read the token's logit by now)
      zero_range<THREADS, DT>(grow, lo, hi);
      __syncthreads();
    }
    if (!zero)
      for (int i = tid; i < count; i += THREADS)
        E::store(grow, lo + list[i], grad_one<ENT>(list_x[i], g, p.c.hi));
  } else {
    const bool gvec = (reinterpret_cast<uintptr_t>(grow + head * E::kBytes) & 15u) == 0;
    for (int64_t u0 = tid; u0 < n_u; u0 += THREADS * kUnroll) {
      uint32_t bits[kUnroll];
      uint4 w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) bits[k] = zero || u0 + k * THREADS >= n_u ? 0u : bits_of(u0 + k * THREADS);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) w[k] = load(u0 + k * THREADS, bits[k]);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (u0 + k * THREADS >= n_u) break;
        const int64_t j = e_lo + (u0 + k * THREADS) * U;
        float2 x[N];
        E::unpack(w[k], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i].x = bits[k] >> (2 * i) & 1u ? grad_one<ENT>(x[i].x, g, p.c.hi) : 0.f;
          x[i].y = bits[k] >> (2 * i + 1) & 1u ? grad_one<ENT>(x[i].y, g, p.c.hi) : 0.f;
        }
        if (gvec) {
          *reinterpret_cast<uint4*>(grow + j * E::kBytes) = E::pack(x);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            E::store(grow, j + 2 * i, x[i].x);
            E::store(grow, j + 2 * i + 1, x[i].y);
          }
        }
      }
    }
    if (end_j >= 0)
      E::store(grow, end_j, !zero && end_kept ? grad_one<ENT>(E::load(xrow, end_j), g, p.c.hi) : 0.f);
  }
  if constexpr (MANY) {
    __syncthreads();
    many.template write<DT>(p, many_row, slots, grow);
  } else if (in.kept_t && token >= lo && token < hi) {
    __syncthreads();
    if (tid == 0) E::store(grow, token, g.at);
  }
}

// ---------------------------------------------------------------------------
// Tensor memory as plain storage: 256 KB an SM that only tensor-core products
// use otherwise. A thread keeps 32-bit words in its own lane of it: a warp
// reaches the 32 lanes of its number mod 4, so warps that share a quarter take
// different columns. All of these are warp-wide.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(columns)
               : "memory");
}

__device__ __forceinline__ void tmem_waive() {  // this CTA allocates no (more) of it
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

// Counts this thread at another CTA's barrier, and orders nothing (in release
// form it is a fence: policy loss of 1024 x 262144 bf16 179 us against 170).
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 words of every lane to and from 16 columns.
__device__ __forceinline__ void tmem_put(uint32_t addr, const uint4 (&w)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(w[0].x), "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[1].x), "r"(w[1].y), "r"(w[1].z), "r"(w[1].w),
      "r"(w[2].x), "r"(w[2].y), "r"(w[2].z), "r"(w[2].w), "r"(w[3].x), "r"(w[3].y), "r"(w[3].z), "r"(w[3].w)
      : "memory");
}

__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_get(uint32_t addr, uint4 (&w)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z), "=r"(w[1].w),
        "=r"(w[2].x), "=r"(w[2].y), "=r"(w[2].z), "=r"(w[2].w), "=r"(w[3].x), "=r"(w[3].y), "=r"(w[3].z), "=r"(w[3].w)
      : "r"(addr)
      : "memory");
}

// ---------------------------------------------------------------------------
// Sums and gradient with the CTA's share of the row held on the SM in between,
// so that HBM is read once and written once. The share arrives by bulk copies
// (TMA) of kPiece bytes into kSlots slots of shared memory. The last kSlots
// pieces stay there; the ones before them move on to tensor memory as they are
// summed, which frees their slots for the later copies. Eight CTAs on an SM hold
// 448 KB of rows that way (56 KB each: 24 in shared memory, 32 in tensor memory),
// against 216 KB in shared memory alone: while some wait for their cluster's
// sums, the others' copies and stores keep HBM busy.
//
// HBM bounds it: policy loss of 1024 x 262144 bf16 171 us, 6.3 TB/s of reads and
// writes (when it took 170: shared memory alone, three CTAs of 64 KB: 201 us; shares of 64 KB, six
// CTAs: 174; three CTAs of 256 threads and 128 KB: 179). A single wave of blocks
// reads, merges and writes one after another: 255 x 50021 fp32 19 us for 102 MB.
// ---------------------------------------------------------------------------
constexpr int kResThreads = 128;
constexpr int kResBlocks = 8;
constexpr int kPieceUnits = kResThreads * kUnroll;
constexpr int kPiece = kPieceUnits * 16;
constexpr int kSlots = 3;
constexpr int kMoved = 4;  // pieces in tensor memory, at most
constexpr int kTmemColumns = kMoved * 16 * (kResThreads / 128);
constexpr uint64_t kCopyLimitNs = 200ull * 1000 * 1000;
// A CTA keeps its tensor memory this long while its cluster's sums are not all
// there, some 50 times what a share takes. Allocation blocks, so a CTA of the
// cluster can be waiting for columns that another kernel holds, whose own other
// CTAs can be waiting for this CTA's columns. Then the pieces in them are given
// up, and read again for the gradient: no CTA waits for ever with columns held.
// (The watch costs 1 us of 171; with every CTA giving its columns up, 184 us.)
constexpr uint64_t kHoldLimitNs = 1000ull * 1000;

// MOVED: the share has more than kSlots pieces. Tensor memory is taken first
// of all: an SM starts no further block of a kernel that may take some before
// the last one has given up its right to (measured: without that, blocks of
// this kernel ran one after another on an SM, 2.5 times the time).
template <int DT, bool ENT, bool MOVED, bool MANY = false>
__global__ void __launch_bounds__(kResThreads, kResBlocks) resident_kernel(const LossParams p, int op) {
  using E = Elem<DT>;
  constexpr int N = E::kUnit / 2;
  extern __shared__ __align__(128) uint4 units[];
  __shared__ __align__(8) uint64_t bars[kSlots];
  __shared__ StatSlots<kResThreads> slots;
  __shared__ RowGrad grad;
  __shared__ RowIn in;
  __shared__ uint32_t tmem_at;
  __shared__ bool given_up;               // this CTA's tensor memory
  __shared__ __align__(8) uint64_t sent;  // the cluster's CTAs, as they send their sums
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t C = p.C;
  const int64_t row = cluster_id();
  const int64_t token = MANY ? -1 : p.tokens[row];
  const uint32_t rank = C > 1 ? cluster_rank() : 0u;
  const Share<DT> sh(p, row, rank);
  const int n = static_cast<int>(sh.u_hi - sh.u_lo);
  const int pieces = (n + kPieceUnits - 1) / kPieceUnits;
  const int moved = MOVED ? max(0, pieces - kSlots) : 0;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(smem_u32(&bars[i]), 1);
    if (MOVED) {
      mbar_init(smem_u32(&sent), C);
      given_up = false;
    }
    fence_mbar_init();
  }
  RowGrad g = {0.f, 0.f, 0.f, 0.f};
  Many<kResThreads> many;
  // where this thread's ids lie in the share, in bytes: they are read as their pieces
  // land (from HBM, 64 of them a row of 512 x 151936 cost 12 us of 61)
  int many_at[Many<kResThreads>::kEach];
#pragma unroll
  for (int i = 0; i < Many<kResThreads>::kEach; ++i) many_at[i] = -1;
  __shared__ double many_sums[MANY ? kResThreads / 32 : 1], many_ranks[MANY ? kMaxRanks : 1];
  __shared__ ManyRow many_row;
  bool ignored = false;
  if constexpr (MANY) {
    // the first pieces on their way to L2 while the ids and their gradients are read
    if (tid == 0 && n > 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(sh.unit(sh.u_lo)),
                   "r"(static_cast<uint32_t>(min(n, kSlots * kPieceUnits)) * 16u)
                   : "memory");
  }
  if constexpr (MANY)
    ignored = !many.load(p, row, [&](int i, int64_t id) {
      if (!sh.owns(id)) return -INFINITY;
      const int64_t u = id - sh.head - sh.u_lo * E::kUnit;
      if (id < sh.head || id >= sh.head + sh.nu * E::kUnit) return E::load(sh.x, id);
      many_at[i] = static_cast<int>(u) * E::kBytes;
      return -INFINITY;
    });
  else
    ignored = token < 0 || token >= p.V;
  if (ignored) {  // (the same in every CTA of the cluster)
    if (MOVED && warp == 1) tmem_waive();
    if (!MANY && tid == 0 && rank == 0) row_ignored(p, op, nullptr, row);
    write_grad<kResThreads, DT, ENT>(p, sh, row, g, -1);
    return;
  }
  if (C > 1) cluster_arrive_relaxed();  // every CTA of the cluster runs before its memory is written
  const unsigned char* src = static_cast<const unsigned char*>(sh.unit(sh.u_lo));
  auto fill = [&](int i) {
    const uint32_t bytes = static_cast<uint32_t>(min(kPieceUnits, n - i * kPieceUnits)) * 16u;
    const uint32_t bar = smem_u32(&bars[i % kSlots]);
    mbar_expect_tx(bar, bytes);
    bulk_g2s(smem_u32(units + (i % kSlots) * kPieceUnits), src + static_cast<int64_t>(i) * kPiece, bytes, bar);
  };
  if (tid == 0)
    for (int i = 0; i < min(pieces, kSlots); ++i) fill(i);
  if (MOVED && warp == 1) {
    tmem_alloc(smem_u32(&tmem_at), kTmemColumns);
    tmem_waive();
  }
  __syncthreads();  // the barriers are initialised, tensor memory is there
  const uint32_t tmem =
      MOVED ? tmem_at + (static_cast<uint32_t>(warp & 3) << 21) + static_cast<uint32_t>(warp >> 2) * (kMoved * 16) : 0u;
  if (!MANY && tid == 32) in = row_in<DT>(p, op, row, token);  // (read after the sums' barrier)
  float end_x = 0.f;
  int64_t end_j = -1;
  if (sh.ends && tid < Share<DT>::kEnds) end_j = sh.end_index(tid);
  if (end_j >= 0) end_x = E::load(sh.x, end_j);
  Running<ENT> run;
  bool landed = true;
  for (int i = 0; i < pieces; ++i) {
    // a copy that never lands (not expected on a healthy device) gives a row
    // of NaN instead of a hang
    landed = landed && mbar_wait_bounded(smem_u32(&bars[i % kSlots]), (i / kSlots) & 1, kCopyLimitNs);
    landed = __all_sync(kAll, landed);
    const uint4* at = units + (i % kSlots) * kPieceUnits + tid;
    const int left = n - i * kPieceUnits;
    if constexpr (MANY) {
#pragma unroll
      for (int j = 0; j < Many<kResThreads>::kEach; ++j)
        if (many_at[j] >= 0 && many_at[j] / kPiece == i)
          many.x[j] = E::load(units + (i % kSlots) * kPieceUnits, many_at[j] % kPiece / E::kBytes);
    }
    if (left >= kPieceUnits) {
      uint4 w[kUnroll];
      float2 x[kUnroll * N];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) w[k] = at[k * kResThreads];
      if (MOVED && i < moved) {
        tmem_put(tmem + i * 16, w);
        __syncthreads();  // the slot is read
        if (tid == 0 && landed) {
          fence_proxy_async_smem();
          fill(i + kSlots);
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) E::unpack(w[k], reinterpret_cast<float2(&)[N]>(x[k * N]));
      run.add_unit(x, p.c);
    } else {
      for (int u = tid; u < left; u += kResThreads, at += kResThreads) {
        float2 x[N];
        E::unpack(*at, x);
        run.add_unit(x, p.c);
      }
    }
  }
  if (end_j >= 0) run.add_one(end_x, p.c);
  if (!landed) run.s = run.t = NAN;
  if constexpr (MANY) many.add_up(p, row, many_sums);
  if (MOVED) tmem_put_wait();
  put_stat(run, slots);
  __syncthreads();
  Stat st;
  if (warp == 0) st = warp_stat<kResThreads, ENT>(p.c, slots);
  if (C > 1) {
    cluster_wait();
    if (warp == 0) {
      send_stat<ENT>(st, rank, C, slots.ranks);
      if constexpr (MANY) Many<kResThreads>::send(many_sums, rank, C, many_ranks);
      if (MOVED && tid < C) arrive_remote(map_rank(smem_u32(&sent), tid));
    }
    cluster_arrive();
    if (MOVED && warp == 1 &&
        (p.give_back || !__all_sync(kAll, mbar_wait_bounded(smem_u32(&sent), 0, kHoldLimitNs)))) {
      given_up = true;  // (read after a barrier)
      tmem_free(tmem_at, kTmemColumns);
    }
    cluster_wait();
    if (warp == 0) st = merge_ranks<ENT>(C, p.c, slots.ranks);
  } else if constexpr (MANY) {
    if (warp == 0) Many<kResThreads>::send(many_sums, 0u, 1u, many_ranks);
    __syncwarp();
  }
  RowVals v;
  if (tid == 0) {
    if constexpr (MANY) {
      v = row_vals<ENT>(p, RowIn{}, st);
      grad = Many<kResThreads>::template weights<ENT>(p, row, st, v, many_ranks, many_row);
    } else {
      v = row_vals<ENT>(p, in, st);
      grad = row_weights<ENT>(p, op, in, st, v);
    }
  }
  __syncthreads();
  if (!MANY && tid == 0 && rank == 0) row_out<ENT>(p, op, nullptr, row, in, st, v);
  if constexpr (MANY) many.keep(p, row, slots);
  __syncwarp();
  g = grad;
  unsigned char* grow = static_cast<unsigned char*>(p.grad) + row * p.ld_grad * E::kBytes;
  unsigned char* gu = grow + (sh.head + sh.u_lo * E::kUnit) * E::kBytes;
  if (g.a == 0.f && g.h == 0.f) {
    write_grad<kResThreads, DT, ENT>(p, sh, row, g, token);
  } else {
    const float2 nm = both(-g.m), cc = both(p.c.hi), aa = both(g.a), hh = both(g.h);
    auto entries = [&](uint4 w, float2 (&e)[N]) {
      float2 x[N];
      E::unpack(w, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 y = mul2(add2(x[i], nm), cc);
        const float2 w2 = make_float2(ex2(y.x), ex2(y.y));
        e[i] = ENT ? mul2(w2, fma2(hh, make_float2(y.x < kMinExp ? kMinExp : y.x, y.y < kMinExp ? kMinExp : y.y), aa))
                   : mul2(w2, aa);
      }
    };
    const bool vec = (reinterpret_cast<uintptr_t>(gu) & 15u) == 0;
    auto put = [&](int u, const float2 (&e)[N]) {
      if (vec) {
        reinterpret_cast<uint4*>(gu)[u] = E::pack(e);
      } else {  // gradient rows aligned otherwise than the logits': entry by entry
#pragma unroll
        for (int k = 0; k < N; ++k) {
          E::store(gu, static_cast<int64_t>(u) * E::kUnit + 2 * k, e[k].x);
          E::store(gu, static_cast<int64_t>(u) * E::kUnit + 2 * k + 1, e[k].y);
        }
      }
    };
    for (int i = 0; i < pieces; ++i) {
      const uint4* at = units + (i % kSlots) * kPieceUnits + tid;
      const int u0 = i * kPieceUnits + tid;
      if (n - i * kPieceUnits >= kPieceUnits) {
        uint4 w[kUnroll];
        if (MOVED && i < moved) {
          if (!given_up) {
            tmem_get(tmem + i * 16, w);
          } else {
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) w[k] = __ldcs(reinterpret_cast<const uint4*>(src) + u0 + k * kResThreads);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kUnroll; ++k) w[k] = at[k * kResThreads];
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
          float2 e[N];
          entries(w[k], e);
          put(u0 + k * kResThreads, e);
        }
      } else {
        for (int u = u0; u < n; u += kResThreads, at += kResThreads) {
          float2 e[N];
          entries(*at, e);
          put(u, e);
        }
      }
    }
    if (end_j >= 0) E::store(grow, end_j, grad_one<ENT>(end_x, g, p.c.hi));
    if (!MANY && sh.owns(token)) {
      __syncthreads();
      if (tid == 0) E::store(grow, token, g.at);
    }
  }
  if constexpr (MANY) {
    __syncthreads();
    many.template write<DT>(p, many_row, slots, grow);
  }
  if (MOVED) {
    __syncthreads();  // every warp has read its words
    if (warp == 1 && !given_up) tmem_free(tmem_at, kTmemColumns);
  }
  if (!landed) {
    // (bounded) copies in flight end before this CTA's memory is given up
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kCopyLimitNs) __nanosleep(1000);
  }
}

// *out = sum of w[i] v[i] by one block of N threads in one fixed order, in
// fp64 (w null: 1 / n). v are the values as they are given out, rounded to fp32
// (their own errors are as large as that: 3e-8 of a row of a policy loss). A weight of 0 takes nothing of a value that has left
// fp32 (0, not 0 * inf); NaN stays. slots: N / 32 doubles of shared memory.
template <int N>
__device__ __forceinline__ void weighted_sum(const float* v, const float* w, int64_t n, float* out, double* slots) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += N) {
    const float x = v[i], weight = w != nullptr ? w[i] : 1.f;
    s += weight == 0.f && isinf(x) ? 0.0 : static_cast<double>(x) * weight;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = threadIdx.x < N / 32 ? slots[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (threadIdx.x == 0) *out = n == 0 ? 0.f : static_cast<float>(w != nullptr ? s : s / static_cast<double>(n));
  }
}

constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) weighted_sum_kernel(const float* v, const float* w, int64_t n, float* out) {
  __shared__ double slots[kSumThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  weighted_sum<kSumThreads>(v, w, n, out, slots);
}

// ---------------------------------------------------------------------------
// Preference loss: the rows' sums, the pairs, the rows' gradient, a kernel
// each. The gradient needs the sums of both sequences of its pair, so logits are
// read twice. (Measured and not kept: one persistent kernel that takes a pair's
// gradient right after its sums, for its second reads to hit L2, 1.6 to 2 times
// the time, as every share then ends in a fence and an atomic; rows that wait on
// the SM for their pair and write without a second read, 1.3 to 1.5 times, as
// every row then ends in a fence and an atomic and the SMs idle at a pair's end.)
// ---------------------------------------------------------------------------

// log(1 + e^x), x = hi + lo, and the sigmoid.
__device__ __forceinline__ float softplus(float hi, float lo) {
  return fmaxf(hi, 0.f) + (hi > 0.f ? lo : 0.f) + log1pf(expf(-fabsf(hi)) * (1.f - copysignf(1.f, hi) * lo));
}
__device__ __forceinline__ float sigmoid(float hi, float lo) {
  const float e = expf(-hi), r = 1.f / (1.f + e);
  return e < INFINITY ? fmaf(lo * r, e * r, r) : expf(hi) * (1.f + lo);  // its slope is r (1 - r)
}

constexpr int kPairThreads = 256;

// One CTA per pair, and one more: the two sequences' sums in a fixed order, the
// pair's loss, and the gradient weights of its rows; the last CTA has the rows
// that no sequence owns.
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const LossParams p, const PrefParams q,
                                                            const RowStat* stats, RowGrad* grads) {
  __shared__ double slots[kPairThreads / 32][4];
  __shared__ float slope[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = blockIdx.x;
  const int tid = threadIdx.x;
  const int32_t B = static_cast<int32_t>(p.B);
  // within [0, B] and in order within the pair, whatever starts holds
  int32_t at[3] = {0, 0, 0};
  for (int k = 0; k < 3; ++k)
    if (2 * i + k <= 2 * q.P && q.P > 0) at[k] = min(max(q.starts[2 * i + k], k > 0 ? at[k - 1] : 0), B);
  auto outside = [&](int64_t row) {
    if (p.logp != nullptr) p.logp[row] = 0.f;
    if (p.grad != nullptr) grads[row] = RowGrad{0.f, 0.f, 0.f, 0.f};
  };
  if (i >= q.P) {
    const int32_t lo = q.P > 0 ? min(max(q.starts[0], 0), B) : B;
    for (int64_t row = tid; row < lo; row += kPairThreads) outside(row);
    for (int64_t row = max(at[0], lo) + tid; row < p.B; row += kPairThreads) outside(row);
    return;
  }
  // sums of logp and numbers of rows of both sequences at once
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  RowStat mine = {0.0, 0.f, -1.f};  // this thread's first row
  for (int64_t row = at[0] + tid; row < at[2]; row += kPairThreads) {
    const RowStat st = stats[row];
    if (row < at[0] + kPairThreads) mine = st;
    if (st.s < 0.f) continue;
    const int k = row < at[1] ? 0 : 2;
    v[k] += st.logp;
    v[k + 1] += 1.0;
  }
  float ref[2] = {0.f, 0.f}, wt = q.inv_p;
  if (tid == 0) {
    if (q.ref != nullptr) {
      ref[0] = q.ref[2 * i];
      ref[1] = q.ref[2 * i + 1];
    }
    if (q.weights != nullptr) wt = q.weights[i];
    if (p.grad_loss != nullptr) wt *= *p.grad_loss;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += __shfl_xor_sync(kAll, v[k], o);
  if ((tid & 31) < 4) slots[tid >> 5][tid & 31] = v[tid & 3];
  __syncthreads();
  if (tid == 0) {
    double ratio = 0.0;
    float scale[2];
    for (int k = 0; k < 2; ++k) {
      double sum = 0.0, n = 0.0;
      for (int x = 0; x < kPairThreads / 32; ++x) {
        sum += slots[x][2 * k];
        n += slots[x][2 * k + 1];
      }
      const double one = q.length_norm && n > 0.0 ? 1.0 / n : 1.0;
      sum *= one;
      scale[k] = static_cast<float>(one);
      q.seq_logp[2 * i + k] = static_cast<float>(sum);
      ratio += k == 0 ? sum - ref[0] : ref[1] - sum;
    }
    const double z = q.beta * ratio - q.margin;
    const float zh = static_cast<float>(z), zl = isfinite(zh) ? static_cast<float>(z - zh) : 0.f;
    const float ls = static_cast<float>(q.smoothing), keep = static_cast<float>(1.0 - q.smoothing);
    float d = -keep * sigmoid(-zh, -zl);
    if (ls != 0.f) d = fmaf(ls, sigmoid(zh, zl), d);
    d = d * wt * q.beta_parts[0] * q.beta_parts[1];
    slope[0] = d * scale[0];
    slope[1] = -d * scale[1];
    q.log_ratio[i] = static_cast<float>(ratio);
    float loss = keep != 0.f ? keep * softplus(-zh, -zl) : 0.f;
    if (ls != 0.f) loss = fmaf(ls, softplus(zh, zl), loss);
    q.pair_loss[i] = z != z ? zh : loss;
  }
  if (p.grad == nullptr) return;
  __syncthreads();
  for (int64_t row = at[0] + tid; row < at[2]; row += kPairThreads) {
    const RowStat st = row < at[0] + kPairThreads ? mine : stats[row];
    RowGrad g = {0.f, 0.f, 0.f, 0.f};
    if (!(st.s < 0.f))
      g = row_grad(slope[row < at[1] ? 0 : 1], 0.f, static_cast<float>(st.logp), 0.f, 0.f, st.m, st.s, p.inv_t);
    grads[row] = g;
  }
}

// The gradient of every row, the last rows first: those are the ones the sums'
// kernel has left in L2 (of 300 x 128256 bf16, 77 MB, 56 MB are still there). The
// first CTA adds up the loss. HBM bounds it: 1222 x 201088 bf16 in 146 us is
// 6.7 TB/s of reads and writes.
template <int DT>
__global__ void __launch_bounds__(kLossThreads, kLossBlocks) pref_grad_kernel(const LossParams p, const PrefParams q,
                                                                              const RowGrad* grads) {
  __shared__ double slots[kLossThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = p.B - 1 - blockIdx.x / p.C;
  const RowGrad g = grads[row];
  const int64_t token = p.tokens[row];
  if (blockIdx.x == 0) weighted_sum<kLossThreads>(q.pair_loss, q.weights, q.P, p.loss, slots);
  const Share<DT> sh(p, row, blockIdx.x % p.C);
  write_grad<kLossThreads, DT, false>(p, sh, row, g, token < p.V ? token : -1);
}

// p for C CTAs a row, which share its units of so many elements.
LossParams with_ctas(const LossParams& p, int64_t unit, uint32_t C) {
  LossParams q = p;
  const int64_t units = p.V / unit;
  q.C = C;
  q.per = (units + C - 1) / C;
  return q;
}

constexpr int64_t kResidentUnits = static_cast<int64_t>(kSlots + kMoved) * kPieceUnits;  // a share's, at most

// CTAs per row for resident_kernel (0: a row does not fit in a cluster): as
// few as hold the row, and more where the batch leaves SMs idle. More than that
// cost merges (policy loss of 1024 x 262144 bf16: 10 CTAs 171 us, 12 CTAs 181, 16
// CTAs 202; gradients of 1000 x 16000 bf16 from HBM: 1 CTA 20.5 us, 2 CTAs 22.5, 4
// CTAs 28.7).
uint32_t resident_ctas(const LossParams& p, int dtype) {
  const int64_t units = p.V / (dtype == QRITA_DTYPE_F32 ? 4 : 8);
  const int64_t least = units > 0 ? (units + kResidentUnits - 1) / kResidentUnits : 1;
  if (least > kMaxRanks || p.B * least > INT32_MAX) return 0;
  int64_t C = static_cast<int64_t>(device_sms()) * kResBlocks / p.B;
  if (C > units / 256) C = units / 256;
  if (C > kMaxRanks) C = kMaxRanks;
  return static_cast<uint32_t>(C > least ? C : least);
}

template <int DT, bool ENT, bool MANY>
cudaError_t launch_resident(const LossParams& p, int op, uint32_t C, cudaStream_t st) {
  const LossParams q = with_ctas(p, Elem<DT>::kUnit, C);
  if (q.per > kResidentUnits) return cudaErrorInvalidValue;  // (a share past its storage)
  const int64_t pieces = (q.per + kPieceUnits - 1) / kPieceUnits;
  const size_t smem = static_cast<size_t>(pieces < kSlots ? pieces : kSlots) * kPiece;
  static_assert(kSlots * kPiece <= 40 * 1024, "a kernel that does not ask has 48 KB, static memory included");
  auto* fn = pieces > kSlots ? &resident_kernel<DT, ENT, true, MANY> : &resident_kernel<DT, ENT, false, MANY>;
  return launch(fn, static_cast<unsigned>(p.B * C), kResThreads, C, st, smem, q, op);
}

template <int DT, bool ENT, bool MANY = false>
cudaError_t launch_rows_of(const LossParams& p, int op, RowStat* stats, cudaStream_t st) {
  if (p.mask != nullptr) {
    // a share's bits fit in the map: with one CTA a row instead of two, the rows
    // of 262144 that keep many leave a tail (the mixed batch above: 313 us), where
    // the sets of 64 alone are faster (47 us against 53)
    uint32_t C = row_ctas(p.B, p.V, false, kLossBlocks);
    while (C < kMaxRanks && p.V / C > kKeptMap<kLossThreads> && p.B * 2 * C <= INT32_MAX) C *= 2;
    const unsigned grid = static_cast<unsigned>(p.B * C);
    if (C == 1 && p.V <= kShortRow)
      return launch(&kept_kernel<kLossThreads / 2, DT, ENT, MANY>, grid, kLossThreads / 2, C, st, size_t(0),
                    with_ctas(p, kKeptUnit, C), op);
    return launch(&kept_kernel<kLossThreads, DT, ENT, MANY>, grid, kLossThreads, C, st, size_t(0), with_ctas(p, kKeptUnit, C), op);
  }
  if (p.grad != nullptr) {
    const uint32_t C = resident_ctas(p, DT);
    if (C > 0) return launch_resident<DT, ENT, MANY>(p, op, C, st);
  }
  const int64_t bytes = p.V * Elem<DT>::kBytes;
  const uint32_t C = row_ctas(p.B, bytes, p.grad != nullptr, kLossBlocks);
  const unsigned grid = static_cast<unsigned>(p.B * C);
  const LossParams q = with_ctas(p, Elem<DT>::kUnit, C);
  if (C == 1 && bytes <= kShortRow)
    return launch(&row_kernel<kLossThreads / 2, DT, ENT, MANY>, grid, kLossThreads / 2, C, st, size_t(0), q, stats, op);
  return launch(&row_kernel<kLossThreads, DT, ENT, MANY>, grid, kLossThreads, C, st, size_t(0), q, stats, op);
}

cudaError_t launch_rows(const LossParams& p, int dtype, int op, bool ent, RowStat* stats, cudaStream_t st) {
  if (dtype == QRITA_DTYPE_F32)
    return ent ? launch_rows_of<QRITA_DTYPE_F32, true>(p, op, stats, st)
               : launch_rows_of<QRITA_DTYPE_F32, false>(p, op, stats, st);
  return ent ? launch_rows_of<QRITA_DTYPE_BF16, true>(p, op, stats, st)
             : launch_rows_of<QRITA_DTYPE_BF16, false>(p, op, stats, st);
}

cudaError_t launch_sum(const float* v, const float* w, int64_t n, float* out, cudaStream_t st) {
  return launch(&weighted_sum_kernel, 1u, kSumThreads, 1u, st, size_t(0), v, w, n, out);
}

}  // namespace

int launch_logprobs(const LossParams& p, int dtype, qrita_stream_t stream) {
  return static_cast<int>(
      launch_rows(p, dtype, kOpLogprobs, p.entropy != nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

int launch_logprobs_grad(const LossParams& p, int dtype, qrita_stream_t stream) {
  return static_cast<int>(
      launch_rows(p, dtype, kOpGrad, p.g_entropy != nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream)));
}

int launch_scores_grad(const LossParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool ent = p.g_entropy != nullptr;
  if (dtype == QRITA_DTYPE_F32)
    return static_cast<int>(ent ? launch_rows_of<QRITA_DTYPE_F32, true, true>(p, kOpGrad, nullptr, st)
                                : launch_rows_of<QRITA_DTYPE_F32, false, true>(p, kOpGrad, nullptr, st));
  return static_cast<int>(ent ? launch_rows_of<QRITA_DTYPE_BF16, true, true>(p, kOpGrad, nullptr, st)
                              : launch_rows_of<QRITA_DTYPE_BF16, false, true>(p, kOpGrad, nullptr, st));
}

int launch_policy(const LossParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.B > 0) {
    const cudaError_t e =
        launch_rows(p, dtype, kOpPolicy, p.entropy != nullptr || p.entropy_coef != 0.0, nullptr, st);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  return static_cast<int>(launch_sum(p.row_loss, p.weights, p.B, p.loss, st));
}

// Workspace: RowStat[B], then RowGrad[B].
size_t pref_workspace_bytes(int64_t B) {
  const size_t n = static_cast<size_t>(B) * (sizeof(RowStat) + sizeof(RowGrad));
  return n < 256 ? 256 : (n + 255) / 256 * 256;
}

int launch_preference(const LossParams& p, const PrefParams& q, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  RowStat* stats = static_cast<RowStat*>(q.workspace);
  RowGrad* grads = reinterpret_cast<RowGrad*>(stats + p.B);
  PrefParams f = q;
  f.inv_p = q.P > 0 ? static_cast<float>(1.0 / static_cast<double>(q.P)) : 0.f;
  cudaError_t e = cudaSuccess;
  if (p.B > 0) {
    LossParams sums = p;
    sums.grad = nullptr;
    if ((e = launch_rows(sums, dtype, kOpPrefStats, false, stats, st)) != cudaSuccess) return static_cast<int>(e);
  }
  e = launch(&pair_kernel, static_cast<unsigned>(q.P + 1), kPairThreads, 1u, st, size_t(0), p, f,
             static_cast<const RowStat*>(stats), grads);
  if (e != cudaSuccess) return static_cast<int>(e);
  if (p.B == 0 || p.grad == nullptr) return static_cast<int>(launch_sum(q.pair_loss, q.weights, q.P, p.loss, st));
  const int bytes = dtype == QRITA_DTYPE_F32 ? 4 : 2;
  const uint32_t C = row_ctas(p.B, p.V * bytes, true, kLossBlocks);
  auto* fn = dtype == QRITA_DTYPE_F32 ? &pref_grad_kernel<QRITA_DTYPE_F32> : &pref_grad_kernel<QRITA_DTYPE_BF16>;
  return static_cast<int>(launch(fn, static_cast<unsigned>(p.B * C), kLossThreads, 1u, st, size_t(0),
                                 with_ctas(p, 16 / bytes, C), f, static_cast<const RowGrad*>(grads)));
}

}  // namespace qrita
