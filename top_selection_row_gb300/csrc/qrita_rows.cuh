// Softmax sums over rows of logits, shared by the losses' and the scores' kernels:
// element access, a thread's running sums, their merges over a CTA and a cluster,
// and the launch of clusters of CTAs over rows.
//
// With c = log2(e) * inv_temperature and m a kept logit within an octave of weight
// (1 / c) of the largest, a kept logit weighs e_j = 2^y_j, y_j = (x_j - m) c, and
//   S = sum e_j,  T = sum e_j y_j,
//   logp_t = ln2 (y_t - log2 S),  H = ln2 (log2 S - T / S),  p_j = e_j / S.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "qrita_device.cuh"
#include "qrita_losses.h"

namespace qrita {
namespace {

using namespace dev;

constexpr int kLossThreads = 256;
constexpr int kLossBlocks = 4;  // on an SM
constexpr uint32_t kAll = 0xffffffffu;
constexpr double kLn2 = 0.69314718055994530942;
// Exponents below this give weights of 0 in fp32; the clamp keeps products
// of such a weight with its exponent (an entropy's terms) from being 0 * inf.
constexpr float kMinExp = -1000.0f;

// The hardware's base-2 exponential is exact at 0 and lies low by 5.0e-8 of
// its value on average over (-32, -1) (measured over 2^20 arguments, the same
// to 1e-9 in every octave from -1 down; root mean square 5.8e-8), by 2.3e-8 above
// -1, and by nothing above 0. Sums that are shifted by an exponential take its mean
// back. The weights themselves are relative to their thread's (or list's) maximum,
// and most of their sum lies within two octaves of it: S takes back 2.5e-8 of what
// is beside the maximum. (Mean error of logp over peaked and normal rows of 1246 to
// 128256 at temperatures 1 and 0.7: -1.4e-8 to 1.2e-8; taking back 5.0e-8, -3.8e-8
// to -4e-9. It adds up over the rows of a sequence.)
constexpr float kExLow = 5.0e-8f;
constexpr float kExNear = 2.5e-8f;
// The same of a factor 2^d that shifts a sum (d <= 0): 2.3e-8 above -1.
__device__ __forceinline__ float shift_low(float d) { return d > -1.f ? 2.3e-8f : kExLow; }

// Rows this short (bytes that their sums read) take blocks of half the threads
// where a block has one whole: more of them on an SM cover the chain of steps
// that every row goes through. Log-probabilities of 4000 rows of 2000, 8000 and
// 16000 bf16: 8.6, 13.7 and 26.1 us against 13.2, 18.8 and 32.6; of 700 rows of
// 32000 (64 KB), from HBM, 18.4 us against 16.4.
constexpr int64_t kShortRow = 32 * 1024;

// The softmax sums of some of a row's kept logits, relative to one of them, m,
// within an octave of the largest (-inf, and sums of 0, before the first): S and
// T as fp32 pairs.
struct Stat {
  float m;
  F2 s, t;
};  // (five words, in this order)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// This CTA's cluster (a CTA alone is a cluster of one).
__device__ __forceinline__ uint32_t cluster_id() {
  uint32_t r;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// The largest of three, NaNs ignored, in one instruction.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// d c for the sums' exponents. c in fp32 is off by up to 6e-8 of itself, the same
// way for every logit of a row, and alone would leave logp off by that of the
// token's distance from the row's mean exponent (1.1e-6 at a distance of 20), and H
// by that of the variance of log p. A single difference takes c as a pair. A group
// of logits takes the low part's product of its largest one, as the addend of its
// multiplications: what is left is the low part's of the distances within a group,
// where a thirty-second of the weight goes three below its top. (The low part of
// each difference by itself, one more instruction a pair: log-probabilities of 4000
// x 8000 bf16 15.7 us against 14.1, of 1024 x 262144 with entropies 91 against 88.)
// The bound, at a weight of 0, keeps what is
// added below 2^-14: an exponent of -inf stays so.
__device__ __forceinline__ float scaled(float d, const Scale& c) { return fmaf(d, c.hi, fmaxf(d, c.bottom) * c.lo); }

// Element access. A row is worked on in units of 16 bytes, aligned in memory:
// `head` elements before the first unit, then the units, then a tail.
template <int DT>
struct Elem;

template <>
struct Elem<QRITA_DTYPE_F32> {
  static constexpr int kBytes = 4;
  static constexpr int kUnit = 4;
  __device__ static float load(const void* row, int64_t j) { return static_cast<const float*>(row)[j]; }
  __device__ static void store(void* row, int64_t j, float g) { static_cast<float*>(row)[j] = g; }
  __device__ static void unpack(uint4 v, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static uint4 pack(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
};

// Two fp32 values as a word of two bf16, to nearest even: the one rounding of
// a bf16 gradient.
__device__ __forceinline__ uint32_t bf16_pair(float2 v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}

template <>
struct Elem<QRITA_DTYPE_BF16> {
  static constexpr int kBytes = 2;
  static constexpr int kUnit = 8;
  __device__ static float load(const void* row, int64_t j) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const unsigned short*>(row)[j]) << 16);
  }
  __device__ static void store(void* row, int64_t j, float g) {
    static_cast<unsigned short*>(row)[j] = static_cast<unsigned short>(bf16_pair(make_float2(g, 0.f)));
  }
  __device__ static void unpack(uint4 v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ static uint4 pack(const float2 (&x)[4]) {
    return make_uint4(bf16_pair(x[0]), bf16_pair(x[1]), bf16_pair(x[2]), bf16_pair(x[3]));
  }
};

__device__ __forceinline__ uint4 load_unit(const void* p) { return *static_cast<const uint4*>(p); }

// One CTA's share of a row: units [u_lo, u_hi) of nu, and on rank 0 the head
// and the tail too (fewer than a unit each).
template <int DT>
struct Share {
  const unsigned char* x;  // the row's logits
  int64_t V, head, nu, u_lo, u_hi;
  bool ends;               // this CTA has the head and the tail

  template <typename P>
  __device__ Share(const P& p, int64_t row, uint32_t rank) {
    constexpr int U = Elem<DT>::kUnit;
    V = p.V;
    x = static_cast<const unsigned char*>(p.logits) + row * p.ld * Elem<DT>::kBytes;
    head = ((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / Elem<DT>::kBytes;
    if (head > V) head = V;
    nu = static_cast<int64_t>(static_cast<uint64_t>(V - head) / U);
    u_lo = min(nu, static_cast<int64_t>(rank) * p.per);
    u_hi = min(nu, u_lo + p.per);
    ends = rank == 0;
  }

  __device__ const void* unit(int64_t u) const { return x + (head * Elem<DT>::kBytes) + u * 16; }

  // Index of element i of the ends (head first, then tail), or -1 past them.
  __device__ int64_t end_index(int i) const {
    if (i < head) return i;
    const int64_t j = head + nu * Elem<DT>::kUnit + (i - head);
    return j < V ? j : -1;
  }
  static constexpr int kEnds = 2 * (Elem<DT>::kUnit - 1);  // at most

  // Whether element j is this CTA's.
  __device__ bool owns(int64_t j) const {
    const int64_t u = (j - head) / Elem<DT>::kUnit;  // (j < head: 0 or below, an end)
    return j < head || u >= nu ? ends : u >= u_lo && u < u_hi;
  }
};

// A thread's running sums, relative to a reference: the first finite logit, and
// each one that lies more than an octave of weight (a factor of 2) above the last
// reference. So the sums are shifted, by an exponential that is off by its own
// error, at most once an octave, and what such errors make of the older sums
// halves each time. (With every new maximum as the reference, a row that rises
// slowly is shifted at each of its groups: logp of 128256 ascending logits over
// ranges of 0.25 to 4 off by 1.9e-7 to 4.8e-7 root mean square, and by more when
// each of those shifts is put right by the mean; below 1e-7 this way, for 0.3 to
// 0.9 % of the time.) A reference's own weight is exactly 1, so a token that holds
// most of a row keeps the digits of log p: it is a reference, or there is a
// logit with more than half its weight.
//
// S is compensated: where one token holds most of a row, every other group of its
// thread's share rounds at that token's weight (logp of 700 x 128256 fp32, one
// CTA a row, 31 groups and 2 single units a thread: root mean square error 5.5e-8,
// 1.4e-7 without, for 0.5 % of the time). Taking that token's weight out of its
// own group's sum as well would leave 3.6e-8, for 3 to 7 % of the time.
template <bool ENT>
struct Running {
  float ref = 0.f, s = 0.f, t = 0.f;
  float lo = 0.f;           // to be added to s
  float limit = -INFINITY;  // an octave above ref; -inf before the first finite logit

  bool lost = false;        // add_unit's

  __device__ __forceinline__ float m() const { return limit == -INFINITY ? -INFINITY : ref; }
  __device__ __forceinline__ void raise(float x, const Scale& c) {
    // (the first time the sums are 0, or NaN, whatever the factor)
    const float d = fminf(fmaxf(scaled(ref - x, c), kMinExp), 0.f);
    const float f = ex2(d);
    if (ENT) {
      t = (t + d * s) * f;
      t = fmaf(t, kExLow, t);
    }
    s *= f;
    lo = fmaf(lo, f, s * kExLow);
    ref = x;
    limit = x + c.octave;
  }
  __device__ __forceinline__ void add(float e) {
    const float d = e + lo, sum = s + d;
    lo = d - (sum - s);
    s = sum;
  }
  __device__ __forceinline__ void add_one(float x, const Scale& c) {
    if (x > limit) raise(x, c);
    const float y = scaled(x - ref, c);
    const float e = ex2(y);
    add(e);
    if (ENT) t = fmaf(e, fmaxf(y, kMinExp), t);
  }
  // The part of T of pairs that add_unit has summed last.
  template <int N>
  __device__ __forceinline__ void add_exponents(const float2 (&x)[N], const Scale& c) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y0 = scaled(x[i].x - ref, c), y1 = scaled(x[i].y - ref, c);
      sum = fmaf(ex2(y0), fmaxf(y0, kMinExp), sum);
      sum = fmaf(ex2(y1), fmaxf(y1, kMinExp), sum);
    }
    t += sum;
  }
  // N pairs (a power of two): their own sum first, then one addition to the
  // running one. The more pairs, the more independent exponentials follow
  // one test of the maximum, which is returned (NaNs ignored). FUSED: their part of
  // T in two chains of multiply-adds, with no exponent held above the lowest; where a
  // logit of -inf makes that NaN it is left out, `lost` says so, and the caller
  // gives add_exponents the same pairs.
  template <bool FUSED = false, int N>
  __device__ __forceinline__ float add_unit(const float2 (&x)[N], const Scale& c) {
    float top = fmaxf(x[0].x, x[0].y);
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmax3(top, x[i].x, x[i].y);
    if (top > limit) raise(top, c);
    const float2 nr = both(-ref), by = both(c.hi), low = both(fmaxf(top - ref, c.bottom) * c.lo);
    float2 es[N], ts[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 y = fma2(add2(x[i], nr), by, low);
      es[i] = make_float2(ex2(y.x), ex2(y.y));
      if (ENT && !FUSED) ts[i] = mul2(es[i], make_float2(fmaxf(y.x, kMinExp), fmaxf(y.y, kMinExp)));  // (NaN by the weight)
      if (ENT && FUSED) ts[i & 1] = i < 2 ? mul2(es[i], y) : fma2(es[i], y, ts[i & 1]);
    }
    if (ENT && FUSED) {
      const float sum = (ts[0].x + ts[0].y) + (ts[1].x + ts[1].y);
      lost = sum != sum;
      if (!lost) t += sum;
    }
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) {
        es[i] = add2(es[i], es[i + o]);
        if (ENT && !FUSED) ts[i] = add2(ts[i], ts[i + o]);
      }
    add(es[0].x + es[0].y);
    if (ENT && !FUSED) t += ts[0].x + ts[0].y;
    return top;
  }
};

// Sums relative to m raised to `to` (>= m). One factor here holds a CTA's whole
// share of a row, so what its exponent loses to rounding (2^-25 of it and of the
// difference) is put back: with one token far above the rest, logp of 400 x 50021
// fp32 in shares of a sixth is off by 1.0e-7 root mean square without.
template <bool ENT>
__device__ __forceinline__ void stat_shift(Stat& a, float to, const Scale& c) {
  if (a.m == to) return;
  float dh, dl;
  two_sum(a.m, -to, dh, dl);
  const float y = dh * c.hi, d = fmaxf(y, kMinExp);
  const float lost = y > kMinExp ? fmaf(dh, c.hi, -y) + fmaf(dl, c.hi, dh * c.lo) : 0.f;
  const float f = ex2(d), more = fmaf(lost, static_cast<float>(kLn2), shift_low(d));
  if (ENT) {
    a.t = f2_merge(a.t, f2_prod(d, a.s.hi));
    a.t = f2_mul(a.t, f);
    a.t.lo = fmaf(a.t.hi, more, a.t.lo);
  }
  a.s = f2_mul(a.s, f);
  a.s.lo = fmaf(a.s.hi, more, a.s.lo);
  a.m = to;
}

// The sum of a Stat over the first W lanes of a warp (a power of two), in
// every one of those lanes.
template <bool ENT, int W>
__device__ __forceinline__ Stat lanes_stat(Stat v, const Scale& c) {
  float m = v.m;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
  stat_shift<ENT>(v, m, c);
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    v.s = f2_merge(v.s, f2_make(__shfl_xor_sync(kAll, v.s.hi, o), __shfl_xor_sync(kAll, v.s.lo, o)));
    if (ENT) v.t = f2_merge(v.t, f2_make(__shfl_xor_sync(kAll, v.t.hi, o), __shfl_xor_sync(kAll, v.t.lo, o)));
  }
  return v;
}

constexpr int kMaxRanks = 16;

// Shared memory of row_stat.
template <int THREADS>
struct alignas(16) StatSlots {
  float m[THREADS], s[THREADS], lo[THREADS], t[THREADS];
  Stat ranks[kMaxRanks];
};

template <int THREADS, bool ENT>
__device__ __forceinline__ void put_stat(const Running<ENT>& r, StatSlots<THREADS>& slots) {
  slots.m[threadIdx.x] = r.m();
  slots.s[threadIdx.x] = r.s;
  slots.lo[threadIdx.x] = r.lo;
  if (ENT) slots.t[threadIdx.x] = r.t;
}

// The CTA's sums from what every thread has put, by one warp after a barrier:
// merging pairs in every warp first would cost each of them 100 instructions,
// as many as 25 logits a lane take.
template <int THREADS, bool ENT>
__device__ __forceinline__ Stat warp_stat(const Scale& c, const StatSlots<THREADS>& slots) {
  const int lane = threadIdx.x & 31;
  Stat v;
  v.m = -INFINITY;
  v.s = v.t = f2_make(0.f, 0.f);
  float ms[THREADS / 32];
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    ms[i] = slots.m[lane + 32 * i];
    v.m = fmaxf(v.m, ms[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.m = fmaxf(v.m, __shfl_xor_sync(kAll, v.m, o));
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const float d = ms[i] == v.m ? 0.f : fmaxf(scaled(ms[i] - v.m, c), kMinExp);
    const float f = ex2(d), s = slots.s[lane + 32 * i] * f;
    f2_add(v.s, s);
    v.s.lo += slots.lo[lane + 32 * i] * f + (d != 0.f ? s * shift_low(d) : 0.f);
    if (ENT) {
      const float t = fmaf(d, s, slots.t[lane + 32 * i] * f);
      f2_add(v.t, t);
      v.t.lo += d != 0.f ? t * shift_low(d) : 0.f;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.s = f2_merge(v.s, f2_make(__shfl_xor_sync(kAll, v.s.hi, o), __shfl_xor_sync(kAll, v.s.lo, o)));
    if (ENT) v.t = f2_merge(v.t, f2_make(__shfl_xor_sync(kAll, v.t.hi, o), __shfl_xor_sync(kAll, v.t.lo, o)));
  }
  return v;
}

// Stores a CTA's record (the same in every lane of its first warp) in all C
// CTAs of the cluster, a lane each.
template <bool ENT>
__device__ __forceinline__ void send_stat(const Stat& v, uint32_t rank, uint32_t C, Stat* ranks) {
  const uint32_t lane = threadIdx.x & 31;
  if (lane < C) {
    const uint32_t at = map_rank(smem_u32(&ranks[rank]), lane);
    const float rec[5] = {v.m, v.s.hi, v.s.lo, v.t.hi, v.t.lo};
#pragma unroll
    for (int i = 0; i < (ENT ? 5 : 3); ++i) st_dsmem_u32(at + 4 * i, __float_as_uint(rec[i]));
  }
}

template <bool ENT>
__device__ __forceinline__ Stat merge_ranks(uint32_t C, const Scale& c, const Stat* ranks) {
  const int lane = threadIdx.x & (kMaxRanks - 1);
  Stat v = ranks[lane];
  if (lane >= static_cast<int>(C)) {
    v.m = -INFINITY;
    v.s = v.t = f2_make(0.f, 0.f);
  }
  return lanes_stat<ENT, kMaxRanks>(v, c);
}

// The cluster's sums from those the first warp of every CTA has, in that warp.
// (Every CTA of the cluster is running by now.)
template <bool ENT>
__device__ __forceinline__ void cluster_stat(Stat& v, const Scale& c, uint32_t rank, uint32_t C, Stat* ranks) {
  if (C == 1) return;
  if (threadIdx.x < 32) send_stat<ENT>(v, rank, C, ranks);
  cluster_sync_all();
  if (threadIdx.x < 32) v = merge_ranks<ENT>(C, c, ranks);
}

// The row's sums from every thread's of its cluster of C CTAs, valid in the
// first warp of every CTA, which calls `send` before the cluster's barrier.
template <int THREADS, bool ENT, typename F>
__device__ __forceinline__ Stat row_stat(const Running<ENT>& r, const Scale& c, uint32_t rank, uint32_t C,
                                         StatSlots<THREADS>& slots, F send) {
  put_stat(r, slots);
  __syncthreads();
  Stat v;
  if (threadIdx.x < 32) v = warp_stat<THREADS, ENT>(c, slots);
  if (C > 1) cluster_wait();
  if (threadIdx.x < 32) send();
  __syncwarp();
  cluster_stat<ENT>(v, c, rank, C, slots.ranks);
  return v;
}

// ln of a pair >= 2^-126, as a pair: off by about 2^-25 absolutely beside the
// relative error of the pair itself. S = 2^e f with f in [0.7, 1.42):
// e ln2 is exact in its leading part (12 bits of ln2), ln f is below 0.36.
__device__ __forceinline__ F2 ln_pair(F2 s) {
  const uint32_t b = __float_as_uint(s.hi);
  int e = static_cast<int>(b >> 23) - 127;
  float f = __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u);
  if (f > 1.41f) {
    f *= 0.5f;
    ++e;
  }
  const float n = static_cast<float>(e);
  const float rest = logf(f) + fmaf(n, 1.42860682e-6f, __fdividef(s.lo, s.hi));  // ln2 - 0.693145752
  return f2_merge(f2_make(n * 0.693145752f, 0.f), f2_make(rest, 0.f));
}

// ln2 T / S as a pair. T's mean error is taken back here, as S's has been.
__device__ __forceinline__ F2 mean_exponent(F2 s, F2 t) {
  t.lo = fmaf(t.hi, kExNear, t.lo);
  const float q = f2_float(t) / s.hi;
  const float rest = __fdividef(fmaf(-q, s.hi, t.hi) + fmaf(-q, s.lo, t.lo), s.hi);  // (of 2^-24 of q)
  F2 r = f2_mul(f2_make(q, rest), static_cast<float>(kLn2));
  r.lo = fmaf(q, static_cast<float>(kLn2 - static_cast<float>(kLn2)), r.lo);
  return r;
}

// S of a row's merged sums, with the exponentials' mean error beside the maximum
// taken back.
__device__ __forceinline__ F2 sum_of(const Stat& st) {
  return f2_merge(st.s, f2_make((st.s.hi - 1.f) * kExNear, 0.f));
}

// (x - m) inv_t - ln S as a pair.
__device__ __forceinline__ F2 logp_of(float x, float m, F2 ln_s, float inv_t, float inv_t_lo) {
  F2 d;
  two_sum(x, -m, d.hi, d.lo);
  if (fabsf(d.hi) < 1e30f && fabsf(d.hi * inv_t) < 1e30f) {
    F2 y = f2_mul(d, inv_t);
    y.lo = fmaf(d.hi, inv_t_lo, y.lo);
    return f2_sub(y, ln_s);
  }
  return f2_make(d.hi * inv_t - ln_s.hi, 0.f);  // no digit of ln S counts (or -inf, or NaN)
}

// Kept bits of 16 mask bytes: bit 7 of each nonzero byte, gathered into four
// bits a word by one multiply.
__device__ __forceinline__ uint32_t kept_bits(const uint4 m) {
  if ((m.x | m.y | m.z | m.w) == 0u) return 0u;
  const uint32_t w[4] = {m.x, m.y, m.z, m.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t nz = ((((w[i] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w[i]) >> 7) & 0x01010101u;
    bits |= ((nz * 0x01020408u) >> 24) << (4 * i);
  }
  return bits;
}

constexpr int kUnroll = 4;  // units a thread has in flight

// Multiprocessors of the current device.
inline int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs per row: as many as fill the device (a power of two), with at least a
// unit or two for each thread. Fewer leave SMs idle (log-probabilities of 64 x
// 128256 bf16 from HBM: 8 CTAs 12.3 us, 2 CTAs 16.4, 1 CTA 20.5), more than fill
// it only add merges (300 x 128256 fp32: 2 CTAs 26.9 us, 1 CTA 31.1, 4 CTAs 37.7). When a second pass
// follows, shares of 64 KB at most, so that the rows in flight fit in L2.
inline uint32_t row_ctas(int64_t B, int64_t bytes, bool second_pass, int per_sm) {
  const int sms = device_sms();
  const int64_t slots = static_cast<int64_t>(sms) * per_sm;
  uint32_t C = 1;
  while (C < kMaxRanks && bytes / (2 * C) >= 4096 && B * 2 * C <= slots) C *= 2;
  if (second_pass)
    while (C < 8 && bytes / C > 64 * 1024 && B * 2 * C <= INT32_MAX) C *= 2;
  return C;
}

// Lets fn have `bytes` of dynamic shared memory, once a device (`done` is fn's own;
// a device past the 64th is asked each time).
template <typename F>
cudaError_t allow_smem(F* fn, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if ((done.load(std::memory_order_relaxed) & bit) != 0ull) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename F, typename... Args>
cudaError_t launch(F* fn, unsigned grid, unsigned block, unsigned cluster, cudaStream_t st, size_t smem, Args... args) {
  if (cluster > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  // the CTAs may be scheduled while the previous kernel of the stream drains;
  // they wait for it (griddepcontrol) before touching memory
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

}  // namespace
}  // namespace qrita
