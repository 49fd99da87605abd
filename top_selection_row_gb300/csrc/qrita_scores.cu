// Scores of given tokens over rows of logits: their log-probabilities, the first
// one's rank, the row's entropy and its top alternatives, in one pass.
//
// Qrita technical summary (gist.science, paper 2602.01518), "Problem
// statement": the candidate set beside the drawn token; what a sampler reports of
// both. The sums are those of the losses (qrita_rows.cuh).
//
// The top N of a row, in the stable descending order, without a second pass: a
// thread keeps the largest logit of each group of units it has summed. The N-th
// largest of the threads' own maxima bounds the N-th largest logit from below (N
// threads have one as large), and only groups whose maximum reaches that bound are
// read again: about N of them, 32 logits each, from L2. What reaches the bound is
// listed as 64-bit keys (logit, then lower id) and put in order by counting, a CTA's
// list by itself, the lists of a cluster by searches in one another. Where ties or
// an unlucky order list more than fits, the groups are walked again in steps, and
// the list is cut to its first N whenever it fills: right for every row, and slower.
//
// The rank counts logits above the token's while they are summed: before the
// token's own unit those above its next lower value (equal ones precede it there),
// behind it those above it; bf16 words two at a time.

#include <cstddef>
#include <cstdint>

#include "qrita_rows.cuh"
#include "qrita_scores.h"

namespace qrita {
namespace {

constexpr int kScoreThreads = kLossThreads;
constexpr int kGroups = 32;     // of a thread, at most
constexpr int kListCap = 1024;  // candidates of a CTA
constexpr int kHits = 512;      // groups read again
constexpr int kMaskGroups = 4096;  // of a CTA under a mask, at most

// Elements of the kernel's units, and the units a thread sums in one step.
template <int DT, bool MASKED>
constexpr int kUnitOf = MASKED ? 16 : Elem<DT>::kUnit;
template <int DT, bool MASKED>
constexpr int kStep = MASKED ? 8 : kUnroll;

// One CTA's units [u_lo, u_hi) of a row, with its head and tail on rank 0. Without
// a mask units are 16 bytes of logits, aligned; under one they are 16 ids, aligned
// in the mask, whose logits may lie anywhere.
template <int DT, bool MASKED>
struct Span {
  using E = Elem<DT>;
  static constexpr int U = kUnitOf<DT, MASKED>;
  static constexpr int kEnds = 2 * (U - 1);  // at most
  const unsigned char* x;
  const uint8_t* keep;
  int64_t V, head, nu, u_lo, u_hi;
  bool ends, vec;

  __device__ Span(const ScoreParams& p, int64_t row, uint32_t rank) {
    V = p.V;
    x = static_cast<const unsigned char*>(p.logits) + row * p.ld * E::kBytes;
    keep = MASKED ? p.mask + row * V : nullptr;
    const uintptr_t at = reinterpret_cast<uintptr_t>(MASKED ? keep : x);
    head = min(V, static_cast<int64_t>(((16u - (at & 15u)) & 15u) / (MASKED ? 1 : E::kBytes)));
    nu = static_cast<int64_t>(static_cast<uint64_t>(V - head) / U);
    u_lo = min(nu, static_cast<int64_t>(rank) * p.per);
    u_hi = min(nu, u_lo + p.per);
    ends = rank == 0;
    vec = (reinterpret_cast<uintptr_t>(x + head * E::kBytes) & 15u) == 0;
  }

  __device__ int64_t id(int64_t u) const { return head + u * U; }
  __device__ int64_t end_index(int i) const {
    if (i < head) return i;
    const int64_t j = head + nu * U + (i - head);
    return j < V ? j : -1;
  }
  __device__ bool kept(int64_t j) const { return !MASKED || keep[j] != 0; }
  __device__ float value(int64_t j) const { return kept(j) ? E::load(x, j) : -INFINITY; }

  // The kept bits of a unit (all of an unmasked one).
  __device__ uint32_t bits(int64_t u) const { return MASKED ? kept_bits(load_unit(keep + id(u))) : 0xFFFFu; }
  // The words of a unit's logits; nothing is read where no bit is set.
  static constexpr int W = U * E::kBytes / 16;
  __device__ void words(int64_t u, uint32_t b, uint4 (&w)[W]) const {
    const int64_t j = id(u);
    if (MASKED && b == 0u) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    } else if (!MASKED || vec) {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = load_unit(x + j * E::kBytes + 16 * i);
    } else {
      float2 v[U / 2];
#pragma unroll
      for (int i = 0; i < U / 2; ++i) {
        v[i].x = b >> (2 * i) & 1u ? E::load(x, j + 2 * i) : 0.f;
        v[i].y = b >> (2 * i + 1) & 1u ? E::load(x, j + 2 * i + 1) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = E::pack(reinterpret_cast<const float2(&)[E::kUnit / 2]>(v[i * E::kUnit / 2]));
    }
  }
  // Their values, -inf where they are not kept.
  __device__ static void expand(const uint4 (&w)[W], uint32_t b, float2* v) {
#pragma unroll
    for (int i = 0; i < W; ++i) E::unpack(w[i], reinterpret_cast<float2(&)[E::kUnit / 2]>(v[i * E::kUnit / 2]));
    if (MASKED) {
#pragma unroll
      for (int i = 0; i < U / 2; ++i) {
        if (!(b >> (2 * i) & 1u)) v[i].x = -INFINITY;
        if (!(b >> (2 * i + 1) & 1u)) v[i].y = -INFINITY;
      }
    }
  }
};

// Larger for logits that come first in the stable descending order.
__device__ __forceinline__ unsigned long long order_key(float x, int64_t id) {
  return static_cast<unsigned long long>(f2key(x)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

// 1.0 in each half where a > b, and the sum of two such words.
__device__ __forceinline__ uint32_t bf2_gt(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t bf2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What counts the logits that precede the first token: those above `at`, and above
// `below` in units before its own. (bf16: both values twice in a word.)
struct Above {
  float at, below;
  uint32_t at2, below2;
  int unit;  // the token's, of this CTA's: -1 before its first, the number of them behind its last
};

template <int DT>
__device__ __forceinline__ Above above_of(float x) {
  Above a;
  a.at = x;
  // the next lower value of the type (x is finite; below +-0 the largest negative one)
  uint32_t b = __float_as_uint(x);
  if (DT == QRITA_DTYPE_BF16) b >>= 16;
  const uint32_t sign = DT == QRITA_DTYPE_BF16 ? 0x8000u : 0x80000000u;
  if ((b & ~sign) == 0u)
    b = sign | 1u;
  else
    b = (b & sign) != 0u ? b + 1u : b - 1u;
  a.below = __uint_as_float(DT == QRITA_DTYPE_BF16 ? b << 16 : b);
  a.at2 = (__float_as_uint(a.at) >> 16) * 0x10001u;
  a.below2 = (__float_as_uint(a.below) >> 16) * 0x10001u;
  return a;
}

// The first n of the c listed keys, largest first, to `first`, by counting the keys
// above each: a few lanes a key while there are few of them. The block is in step.
template <int THREADS>
__device__ __forceinline__ void first_of(const unsigned long long* list, int c, int n, unsigned long long* first) {
  const int parts = c <= THREADS / 8 ? 8 : c <= THREADS / 4 ? 4 : 1;
  const int part = threadIdx.x & (parts - 1);
  for (int i0 = 0; i0 < c; i0 += THREADS / parts) {
    const int i = i0 + threadIdx.x / parts;
    const unsigned long long k = i < c ? list[i] : ~0ull;
    int r = 0;
#pragma unroll 4
    for (int j = part; j < c; j += parts) r += list[j] > k;
    for (int o = 1; o < parts; o <<= 1) r += __shfl_xor_sync(kAll, r, o);
    if (i < c && part == 0 && r < n) first[r] = k;
  }
}

__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// One CTA a row, or a cluster for few rows. HBM bounds the log-probabilities alone
// (1024 x 262144 bf16 82 us, 6.6 TB/s), and issue slots with it the rest: 88 with
// entropies, 90 with the rank besides, 102 with 20 alternatives too, of which 8 are the
// end of the wave: its blocks' steps that read nothing (bound, groups read again,
// order). 4 x 32000 fp32 with 5 alternatives 8.7 us, of latency. Under a mask that keeps
// 256 of 262144 ids 79 us with all of it (268 MB of masks); one that keeps a tenth at
// random 285 (nearly every unit has a bit, and a warp has one load a lane under way).
template <int THREADS, int DT, bool ENT, bool MASKED>
__global__ void __launch_bounds__(THREADS, kLossThreads * kLossBlocks / THREADS) score_kernel(const ScoreParams p) {
  using Sp = Span<DT, MASKED>;
  constexpr int U = Sp::U, K = kStep<DT, MASKED>, W = Sp::W;
  __shared__ StatSlots<THREADS> slots;
  __shared__ __align__(16) float tops[THREADS], quads[THREADS / 4];
  __shared__ unsigned long long list[kListCap];
  __shared__ unsigned long long first[kMaxTop];
  __shared__ unsigned short hits[kHits];
  __shared__ int count, found;
  __shared__ unsigned long long ranked;
  __shared__ uint32_t bound;   // key of what the N-th largest logit is at least
  __shared__ float row_of[6];  // m, S (its sign and NaN), ln S as a pair, H
  extern __shared__ __align__(16) unsigned char dynamic[];
  float* gmax = reinterpret_cast<float*>(dynamic);  // [groups][THREADS]
  uint32_t* group_keys = reinterpret_cast<uint32_t*>(dynamic);  // (under a mask)
  __shared__ int warp_units[MASKED ? THREADS / 32 : 1][64];
  __shared__ unsigned short warp_bits[MASKED ? THREADS / 32 : 1][64];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const uint32_t C = p.C;
  const int64_t row = cluster_id();
  const uint32_t rank = C > 1 ? cluster_rank() : 0u;
  const Sp sp(p, row, rank);
  const int N = p.N;
  if (C > 1) cluster_arrive_relaxed();  // every CTA of the cluster runs before its memory is written
  if (tid == 0) {
    count = found = 0;
    ranked = 0ull;
    bound = 0xFFFFFFFFu;
  }
  const int n = static_cast<int>(sp.u_hi - sp.u_lo);  // (a row has fewer than 2^31 logits)
  // what the first step reads, on its way while the token's logit is looked up
  if constexpr (!MASKED) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (tid + k * THREADS < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(sp.x + sp.id(sp.u_lo + tid + k * THREADS) * Elem<DT>::kBytes));
  }
  int64_t t0 = -1;
  bool counts = false;
  Above ab = {};
  if (p.rank != nullptr) {
    t0 = p.tokens[row * p.M];
    if (t0 >= 0 && t0 < p.V) {
      const float x = sp.value(t0);
      counts = x > -INFINITY && x < INFINITY;
      if (counts) ab = above_of<DT>(x);
      const int64_t u = t0 < sp.head ? -1 : (t0 - sp.head) / U - sp.u_lo;
      ab.unit = static_cast<int>(min(max(u, static_cast<int64_t>(-1)), static_cast<int64_t>(n)));
    }
  }
  // this thread's given token, whose score waits for the sums
  float mine = -INFINITY;
  int32_t my_token = -1;
  if (rank == 0 && tid < p.M) {
    my_token = p.tokens[row * p.M + tid];
    if (my_token >= 0 && my_token < p.V) mine = sp.value(my_token);
  }
  Running<ENT> run;
  float top = -INFINITY, group = -INFINITY;
  uint32_t before = 0u;  // logits that precede the token
  const int steps = (n + THREADS * K - 1) / (THREADS * K);
  int in_group = 0, g = 0;
  const int each = p.group_steps * (MASKED ? 1 : K);  // units of a group
  const int n_groups = MASKED && N > 0 ? (n + each - 1) / each : 0;
  auto summed = [&](float t, bool end) {
    group = fmaxf(group, t);
    if (N > 0 && (++in_group == p.group_steps || end)) {
      gmax[g * THREADS + tid] = group;
      top = fmaxf(top, group);
      group = -INFINITY;
      in_group = 0;
      ++g;
    }
  };
  uint32_t above2 = 0u;
  auto count_up = [&]() {
    if (!MASKED && DT == QRITA_DTYPE_BF16) {
      before += static_cast<uint32_t>(__uint_as_float(above2 << 16)) + static_cast<uint32_t>(__uint_as_float(above2 & 0xFFFF0000u));
      above2 = 0u;
    }
  };
  auto count_above = [&](const uint4& w, const float2* x, int u) {
    if (!MASKED && DT == QRITA_DTYPE_BF16) {
      const uint32_t at = u < ab.unit ? ab.below2 : ab.at2;
      // (1.0 for each half above, added up in bf16: exact up to 256)
      const uint32_t a = bf2_add(bf2_add(bf2_gt(w.x, at), bf2_gt(w.y, at)), bf2_add(bf2_gt(w.z, at), bf2_gt(w.w, at)));
      above2 = bf2_add(above2, a);
    } else {
      const float at = u < ab.unit ? ab.below : ab.at;
#pragma unroll
      for (int i = 0; i < U / 2; ++i) before += (x[i].x > at) + (x[i].y > at);
    }
  };
  if constexpr (MASKED) {
    const uint8_t* keep = sp.keep + sp.id(sp.u_lo);
    // A warp lists its units with a bit set, in their order, and sums them 32 at a time,
    // a lane each: a sparse row's would otherwise be one lane's work after another's.
    // The largest kept logit of each group of neighbouring units is kept as a key.
    const int warp = tid >> 5, lane = tid & 31;
    for (int i = tid; N > 0 && i < n_groups; i += THREADS) group_keys[i] = 0u;
    if (N > 0) __syncthreads();
    int listed = 0;
    auto sum_units = [&](int many) {  // of the warp's list, the first `many`
      if (lane < many) {
        const int u = warp_units[warp][lane];
        const uint32_t b = warp_bits[warp][lane];
        uint4 w[W];
        float2 x[U / 2];
        sp.words(sp.u_lo + u, b, w);
        Sp::expand(w, b, x);
        if (counts) count_above(w[0], x, u);
        const float t = run.add_unit(x, p.c);
        if (N > 0) {
          top = fmaxf(top, t);
          atomicMax(&group_keys[u / each], f2key(t));
        }
      }
    };
    for (int s = 0; s < steps; ++s) {
      const int u0 = s * (THREADS * K) + tid;
      uint4 mw[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        mw[k] = u0 + k * THREADS < n ? __ldcs(reinterpret_cast<const uint4*>(keep) + u0 + k * THREADS) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t b = kept_bits(mw[k]);
        const uint32_t some = __ballot_sync(kAll, b != 0u);
        if (some == 0u) continue;
        if (b != 0u) {
          const int at = listed + __popc(some & ((1u << lane) - 1u));
          warp_units[warp][at] = u0 + k * THREADS;
          warp_bits[warp][at] = static_cast<unsigned short>(b);
        }
        listed += __popc(some);
        __syncwarp();
        if (listed >= 32) {
          sum_units(32);
          __syncwarp();
          listed -= 32;
          int u = 0;
          unsigned short rest = 0;
          if (lane < listed) {
            u = warp_units[warp][32 + lane];
            rest = warp_bits[warp][32 + lane];
          }
          __syncwarp();
          if (lane < listed) {
            warp_units[warp][lane] = u;
            warp_bits[warp][lane] = rest;
          }
          __syncwarp();
        }
      }
    }
    sum_units(listed);
  } else {
    const uint4* units = reinterpret_cast<const uint4*>(sp.x + sp.id(sp.u_lo) * Elem<DT>::kBytes) + tid;
    const int full = n / (THREADS * K);
    auto again = [&](const uint4* at) {
      float2 x[U / 2];
      const uint4 w = load_unit(at);
      Sp::expand(reinterpret_cast<const uint4(&)[1]>(w), 0u, x);
      run.add_exponents(x, p.c);
    };
    for (int s = 0; s < full; ++s, units += THREADS * K) {
      // (L2 is asked for the next step meanwhile: with entropies, rank and 20 alternatives
      // 1024 x 262144 bf16 117 us without, 102 with, 106 for the step after that)
      if (tid == 0 && s + 1 < full)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(units + THREADS * K), "n"(THREADS * K * 16) : "memory");
      uint4 w[K];
      float2 x[K * U / 2];
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] = load_unit(units + k * THREADS);
#pragma unroll
      for (int k = 0; k < K; ++k) Sp::expand(reinterpret_cast<const uint4(&)[1]>(w[k]), 0u, x + k * (U / 2));
      if (counts) {
#pragma unroll
        for (int k = 0; k < K; ++k) count_above(w[k], x + k * (U / 2), s * (THREADS * K) + k * THREADS + tid);
        count_up();
      }
      summed(run.template add_unit<true>(x, p.c), s + 1 == steps);
      if (ENT && run.lost) {  // (logits of -inf)
#pragma unroll 1
        for (int k = 0; k < K; ++k) again(units + k * THREADS);
        run.lost = false;
      }
    }
    if (full < steps) {  // the rest of the units, one at a time
      float t = -INFINITY;
      for (int u = full * (THREADS * K) + tid; u < n; u += THREADS, units += THREADS) {
        float2 x[U / 2];
        const uint4 w = load_unit(units);
        Sp::expand(reinterpret_cast<const uint4(&)[1]>(w), 0u, x);
        if (counts) count_above(w, x, u);
        t = fmaxf(t, run.template add_unit<true>(x, p.c));
        if (ENT && run.lost) again(units);
        run.lost = false;
      }
      count_up();
      summed(t, true);
    }
  }
  // (under a mask a group is `each` neighbouring units, and a column of threads has some)
  const int groups = MASKED ? (n_groups + THREADS - 1) / THREADS : g;
  auto unit_of = [&](int group, int column, int j) {
    return MASKED ? (group * THREADS + column) * each + j : (group * each + j) * THREADS + column;
  };
  auto group_max = [&](int i) {  // of the i-th, NaN where it has none
    if (MASKED) return i < n_groups ? key2f(group_keys[i]) : NAN;
    return gmax[i];
  };
  // the row's head and tail
  int64_t end_j = -1;
  float end_x = -INFINITY;
  if (sp.ends && THREADS - 1 - tid < Sp::kEnds) end_j = sp.end_index(THREADS - 1 - tid);
  if (end_j >= 0) {
    end_x = sp.value(end_j);
    run.add_one(end_x, p.c);
    top = fmaxf(top, end_x);
    if (counts) before += end_x > ab.at || (end_x == ab.at && end_j < t0);
  }
  // equal logits before the token in its own unit
  if (counts && tid == THREADS - 1 && ab.unit >= 0 && ab.unit < n)
    for (int64_t j = sp.id(sp.u_lo + ab.unit); j < t0; ++j) before += sp.value(j) == ab.at;
  put_stat(run, slots);
  // maxima of threads, or (few alternatives) of four threads
  const int maxima = N <= THREADS / 8 ? THREADS / 4 : THREADS;
  if (N > 0) {
    tops[tid] = top;
    if (maxima < THREADS) {
      float t = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      t = fmaxf(t, __shfl_xor_sync(kAll, t, 2));
      if ((tid & 3) == 0) quads[tid >> 2] = t;
    }
  }
  if (p.rank != nullptr) before = __reduce_add_sync(kAll, before);
  __syncthreads();
  if (p.rank != nullptr && (tid & 31) == 0 && before != 0u) atomicAdd(&ranked, static_cast<unsigned long long>(before));
  // the first warp merges the sums while the others look for the alternatives
  Stat st = {};
  auto row_values = [&]() {
    const bool empty = st.s.hi == 0.f;
    const F2 S = sum_of(st);
    const F2 ln_s = empty ? f2_make(0.f, 0.f) : ln_pair(S);
    row_of[0] = st.m;
    row_of[1] = st.s.hi;
    row_of[2] = ln_s.hi;
    row_of[3] = ln_s.lo;
    row_of[4] = ENT && !empty ? f2_float(f2_sub(ln_s, mean_exponent(S, st.t))) : 0.f;
  };
  if (tid < 32) {
    st = warp_stat<THREADS, ENT>(p.c, slots);
    if (C > 1) {
      cluster_wait();
      send_stat<ENT>(st, rank, C, slots.ranks);
    } else if (tid == 0) {
      row_values();
    }
  } else {
    if (C > 1) cluster_wait();
  }
  float least = 0.f;
  auto push = [&](float x, int64_t id) {
    if (x >= least && x > -INFINITY) {
      const int at = atomicAdd(&count, 1);
      if (at < kListCap) list[at] = order_key(x, id);
    }
  };
  if (N > 0 && tid >= 32) {
    constexpr int kOthers = THREADS - 32;
    const int wt = tid - 32;
    auto others_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kOthers) : "memory"); };
    // the N-th largest of the maxima: the least of those with fewer than N above
    const float* of = maxima < THREADS ? quads : tops;
    uint32_t low = 0xFFFFFFFFu;
    for (int i = wt; i < maxima; i += kOthers) {
      const float mine = of[i];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < maxima; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(of + j);
        r += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
      }
      if (r < N) low = min(low, f2key(mine));
    }
    low = __reduce_min_sync(kAll, low);
    if ((tid & 31) == 0 && low != 0xFFFFFFFFu) atomicMin(&bound, low);
    others_sync();
    least = key2f(bound);
    if (end_j >= 0) push(end_x, end_j);
    // the groups that reach it, then their units, each by a thread
    auto hit = [&](float m, int i) {
      if (m >= least && m > -INFINITY) {
        const int at = atomicAdd(&found, 1);
        if (at < kHits) hits[at] = static_cast<unsigned short>(i);
      }
    };
    if (MASKED) {
      for (int i = wt; i < n_groups; i += kOthers) hit(group_max(i), i);
    } else {
      for (int i = wt; i < groups * (THREADS / 4); i += kOthers) {
        const float4 v = reinterpret_cast<const float4*>(gmax)[i];
        hit(v.x, 4 * i);
        hit(v.y, 4 * i + 1);
        hit(v.z, 4 * i + 2);
        hit(v.w, 4 * i + 3);
      }
    }
    others_sync();
    const int tasks = min(found, kHits) * each;
    for (int i = wt; i < tasks; i += kOthers) {
      const int group = hits[i / each];
      const int u = unit_of(group / THREADS, group % THREADS, i % each);
      if (u >= n) continue;
      uint4 w[W];
      float2 x[U / 2];
      const uint32_t b = sp.bits(sp.u_lo + u);
      sp.words(sp.u_lo + u, b, w);
      Sp::expand(w, b, x);
#pragma unroll
      for (int j = 0; j < U / 2; ++j) {
        push(x[j].x, sp.id(sp.u_lo + u) + 2 * j);
        push(x[j].y, sp.id(sp.u_lo + u) + 2 * j + 1);
      }
    }
  }
  int c = 0;
  if (N > 0) {
    __syncthreads();
    c = count;
    if (c > kListCap || found > kHits) {
      // more than fits: again, two logits of a thread at a time, the list cut to its
      // first N whenever the next step might not fit
      __syncthreads();
      if (tid == 0) count = 0;
      unsigned long long above = (static_cast<unsigned long long>(bound) << 32) - 1ull;  // keys beyond it count
      __syncthreads();
      auto put = [&](float x, int64_t id) {
        const unsigned long long key = order_key(x, id);
        if (x > -INFINITY && key > above) list[atomicAdd(&count, 1)] = key;
      };
      auto cut = [&](int room) {
        __syncthreads();
        const int have = count;
        __syncthreads();  // (the next entries change it)
        if (have <= room) return;
        first_of<THREADS>(list, have, N, first);
        __syncthreads();
        for (int i = tid; i < min(have, N); i += THREADS) list[i] = first[i];
        if (tid == 0) count = min(have, N);
        if (have >= N) above = first[N - 1];
        __syncthreads();
      };
      constexpr int kRoom = kListCap - 2 * THREADS;
      if (end_j >= 0) put(end_x, end_j);
      for (int i = 0; i < groups; ++i) {
        const float m = group_max(i * THREADS + tid);
        const bool some = m > -INFINITY && order_key(m, sp.id(sp.u_lo + unit_of(i, tid, 0))) > above;
        if (!__syncthreads_or(some)) continue;
        for (int g = 0; g < each; ++g) {
          const int u = unit_of(i, tid, g);
          const bool mine = some && u < n;
          for (int j = 0; j < U; j += 2) {
            cut(kRoom);
            if (mine) {
              put(sp.value(sp.id(sp.u_lo + u) + j), sp.id(sp.u_lo + u) + j);
              put(sp.value(sp.id(sp.u_lo + u) + j + 1), sp.id(sp.u_lo + u) + j + 1);
            }
          }
        }
      }
      __syncthreads();
      c = count;
    }
    if (tid < N) first[tid] = 0ull;
    __syncthreads();
    first_of<THREADS>(list, c, N, first);
  }
  __syncthreads();
  if (C > 1) {
    cluster_sync_all();  // every CTA's sums, list and count are there
    if (rank != 0) {  // rank 0 reads this CTA's memory until the next barrier
      cluster_arrive_relaxed();
      cluster_wait();
      return;
    }
    if (tid < 32) st = merge_ranks<ENT>(C, p.c, slots.ranks);
    if (p.rank != nullptr && tid > 0 && tid < static_cast<int>(C)) {
      const uint32_t at = map_rank(smem_u32(&ranked), tid);
      const unsigned long long more = static_cast<unsigned long long>(ld_dsmem_u32(at + 4)) << 32 | ld_dsmem_u32(at);
      if (more != 0ull) atomicAdd(&ranked, more);
    }
  }
  if (C > 1 && tid == 0) row_values();
  // The cluster's lists, one after another in the groups' place. With q the smallest
  // number of each list's first entries that makes N together, the least of the q-th
  // entries has N at or above it; what is above is put in order by counting.
  unsigned long long* lists = reinterpret_cast<unsigned long long*>(dynamic);
  if (N > 0 && C > 1) {
    const int all = static_cast<int>(C) * N;
    if (tid >= 32)
      for (int i = tid - 32; i < all; i += THREADS - 32) lists[i] = ld_dsmem_u64(map_rank(smem_u32(&first[i % N]), i / N));
    if (tid == 0) count = 0;
    __syncthreads();
    cluster_arrive();  // (the other CTAs may end)
    const int q = (N + static_cast<int>(C) - 1) / static_cast<int>(C), l = tid & 31;
    unsigned long long low = l < static_cast<int>(C) ? lists[l * N + q - 1] : ~0ull;
#pragma unroll
    for (int o = kMaxRanks / 2; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(kAll, low, o));
    low = max(__shfl_sync(kAll, low, 0), 1ull);
    unsigned long long* merged = lists + all;
    for (int i = tid; i < all; i += THREADS)
      if (lists[i] >= low) merged[atomicAdd(&count, 1)] = lists[i];
    if (tid < N) first[tid] = 0ull;  // (read by nobody else any more)
    __syncthreads();
    first_of<THREADS>(merged, count, N, first);
  } else if (C > 1) {
    cluster_arrive();
  }
  __syncthreads();
  const float m = row_of[0], total = row_of[1];
  const F2 ln_s = f2_make(row_of[2], row_of[3]);
  const bool nan = total != total;
  auto score = [&](float x) {  // of a kept token
    if (nan) return total;
    return total == 0.f || x == -INFINITY ? -INFINITY : f2_float(logp_of(x, m, ln_s, p.inv_t, p.inv_t_lo));
  };
  for (int i = tid; i < p.M; i += THREADS) {
    const int32_t t = i == tid ? my_token : p.tokens[row * p.M + i];
    float lp = 0.f;
    if (t >= 0 && t < p.V) lp = score(i == tid ? mine : sp.value(t));
    p.logp[row * p.M + i] = lp;
  }
  if (tid == 0) {
    // (a finite kept logit has a rank, also where its log p has left fp32)
    if (p.rank != nullptr) p.rank[row] = counts && !nan ? static_cast<int32_t>(ranked) : -1;
    if (ENT) p.entropy[row] = nan ? total : row_of[4];
  }
  if (N > 0) {
    auto put = [&](int at, unsigned long long key) {
      const float x = key2f(static_cast<uint32_t>(key >> 32));
      p.top_ids[row * N + at] = key == 0ull || nan ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
      p.top_logp[row * N + at] = nan ? total : key == 0ull ? -INFINITY : score(x);
    };
    if (tid < N) put(tid, first[tid]);
  }
  if (C > 1) cluster_wait();
}

template <int DT, bool ENT, bool MASKED>
cudaError_t launch_scores_of(const ScoreParams& p, cudaStream_t st) {
  constexpr int U = kUnitOf<DT, MASKED>, K = kStep<DT, MASKED>;
  const int64_t bytes = p.V * (MASKED ? 1 : Elem<DT>::kBytes);
  const int64_t sms = device_sms();
  uint32_t C = 1;
  if (p.N == 0) {
    C = row_ctas(p.B, bytes, false, kLossBlocks);
  } else {
    // Lists to merge cost more than sums: two CTAs an SM with shares of 20 KB (4 KB of a
    // mask), four with 100 KB. (4 x 32000 fp32, 20 alternatives: 4 CTAs a row 9.1 us, 16
    // CTAs 10.3, 2 CTAs 10.0; 64 x 128256 bf16: 4 CTAs 13.0, 8 CTAs 14.9, 2 CTAs 14.6.)
    while (C < kMaxRanks && p.B * 2 * C <= sms * kLossBlocks &&
           bytes / (2 * C) >= (p.B * 2 * C > sms * 2 ? 100000 : MASKED ? 4000 : 20000))
      C *= 2;
  }
  // Blocks of half the threads where rows are short, and where one row a block takes
  // more than a wave: twice as many are on an SM, and a wave ends in the steps of its
  // blocks that read nothing (1024 x 262144 bf16 117 us then, with 256 threads 122). Not
  // for many alternatives: the bound is then that of too few maxima.
  const bool small = C == 1 && (bytes <= kShortRow || (p.N > 0 && p.B > sms * kLossBlocks)) && p.N <= kScoreThreads / 8;
  const int threads = small ? kScoreThreads / 2 : kScoreThreads;
  ScoreParams q = p;
  q.C = C;
  const int64_t units = p.V / U;
  q.per = (units + C - 1) / C;
  const int64_t steps = (q.per + threads * K - 1) / (threads * K);
  q.group_steps = steps <= kGroups ? 1 : static_cast<int>((steps + kGroups - 1) / kGroups);
  if (MASKED) q.group_steps = static_cast<int>((q.per + kMaskGroups - 1) / kMaskGroups > 0 ? (q.per + kMaskGroups - 1) / kMaskGroups : 1);
  size_t smem = 0;
  if (p.N > 0) {
    smem = static_cast<size_t>(MASKED ? (q.per + q.group_steps - 1) / q.group_steps
                                      : (steps + q.group_steps - 1) / q.group_steps * threads) * sizeof(float);
    const size_t lists = static_cast<size_t>(C) * p.N * 16u;
    if (C > 1 && lists > smem) smem = lists;
  }
  static_assert(kGroups * kScoreThreads * 4 + 16 * 1024 <= 48 * 1024, "a kernel that does not ask has 48 KB");
  static_assert(kMaskGroups * 4 <= kMaxRanks * kMaxTop * 16, "groups under a mask fit in what is asked for");
  static_assert(kMaxRanks * kMaxTop * 16 <= kGroups * kScoreThreads * 4, "the lists fit in the groups' place");
  const unsigned grid = static_cast<unsigned>(p.B * C);
  auto go = [&](auto* fn, std::atomic<uint64_t>& done) {
    if (MASKED) {  // (the warps' lists beside the most that the lists of a cluster take)
      const cudaError_t e = allow_smem(fn, kMaxRanks * kMaxTop * 16, done);
      if (e != cudaSuccess) return e;
    }
    return launch(fn, grid, threads, C, st, smem, q);
  };
  static std::atomic<uint64_t> done[2];
  return small ? go(&score_kernel<kScoreThreads / 2, DT, ENT, MASKED>, done[0])
               : go(&score_kernel<kScoreThreads, DT, ENT, MASKED>, done[1]);
}

template <int DT>
cudaError_t launch_scores_type(const ScoreParams& p, cudaStream_t st) {
  if (p.mask != nullptr)
    return p.entropy != nullptr ? launch_scores_of<DT, true, true>(p, st) : launch_scores_of<DT, false, true>(p, st);
  return p.entropy != nullptr ? launch_scores_of<DT, true, false>(p, st) : launch_scores_of<DT, false, false>(p, st);
}

}  // namespace

int launch_scores(const ScoreParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return static_cast<int>(dtype == QRITA_DTYPE_F32 ? launch_scores_type<QRITA_DTYPE_F32>(p, st)
                                                   : launch_scores_type<QRITA_DTYPE_BF16>(p, st));
}

}  // namespace qrita
