// The slots of a key-value cache that a budget keeps: attention weights gathered
// for each slot, the selection of the slots to keep with their rows packed, and a
// full cache's next token put over the slot that is last.
//
// The order of slots is the library's stable descending one (Qrita technical
// summary, gist.science, paper 2602.01518, "Problem statement": the exact result of
// a stable sort), of the weights, with protected slots before all others: the
// kept set is exact, equal weights go to the lower slot.

#include <cstddef>
#include <cstdint>

#include "qrita_cache.h"
#include "qrita_rows.cuh"

namespace qrita {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// Larger for weights that are kept longer: the order of the numbers, NaN below all
// of them (0; -inf's is 0x007FFFFF).
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0u : f2key(w); }

// Every thread of a row's C CTAs. (Without a cluster its barrier is none to rely on:
// threads that arrived at it ahead of others were held there.)
__device__ __forceinline__ void row_sync(uint32_t C) {
  if (C > 1)
    cluster_sync_all();
  else
    __syncthreads();
}

struct Guard {
  int32_t sink;
  int64_t from;  // positions from here on are the last ones seen

  __device__ Guard(const CacheOrder& c, int64_t b, int32_t length) {
    sink = c.sink;
    from = static_cast<int64_t>(c.seen != nullptr ? c.seen[b] : length) - c.recent;
  }
  __device__ bool holds(int32_t position) const { return position < sink || position >= from; }
};

__device__ __forceinline__ int32_t length_of(const CacheOrder& c, int64_t b, int64_t most) {
  return static_cast<int32_t>(min(static_cast<int64_t>(max(c.lengths[b], 0)), most));
}

// ---------------------------------------------------------------------------
// Attention weights.
//
// For one kv head, x_ri = scale q_r . k_i over the rows r (queries, G heads each)
// and visible slots i, and w_i = decay w_i + sum_r exp(x_ri - m_r) / sum_j exp(x_rj - m_r).
// A cluster of CTAs takes a (sequence, kv head), a share of the slots each. First
// every CTA works out its scores and each row's maximum and sum; these merge through
// distributed shared memory; then a slot's weight is the sum over its scores, which
// wait in shared memory where they fit, so that keys are read once, and are worked
// out again from keys that are in L2 where they do not.
//
// HBM bounds it: one query of 4 heads on 16 x 8 x 32768 slots of 128 bf16 196 us (5.5
// TB/s), on 64 x 8 x 4096 94 us (5.7); 4 x 8 x 1024 6.4 us, of latency. A warp has the
// next tile on its way while it works on one, in four chains of products (a single
// chain of 16 dependent ones: 230 us). fp32 keys go by plain loads, a slot a lane: 16 x
// 8 x 8192 slots of 128 211 us (2.5 TB/s).
// ---------------------------------------------------------------------------
constexpr int kWThreads = 256;  // two CTAs on an SM: one's merge beside the other's keys
constexpr int kWWarps = kWThreads / 32;
constexpr int kMaxRowsAtOnce = 32;
// Up to as many rows this kernel takes, which reads keys once; more go to the window's
// where that can be. (32 rows of 64 dimensions in 8 x 8 x 8192 slots: 95 us here, 38
// there; 16 rows of 128 in 64 x 8 x 2000: 77 and 102; 8 in 16 x 8 x 16384: 132 and 173.)
constexpr int kFewRows = 16;

struct alignas(8) RowSum {
  float m, s;
};

__device__ __forceinline__ unsigned long long ld_dsmem_sum(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void sum_add(RowSum& a, RowSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) {  // (sums of 0, or NaN)
    a.s += b.s;
    return;
  }
  a.s = a.s * ex2((a.m - m) * kLog2e) + b.s * ex2((b.m - m) * kLog2e);
  a.m = m;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Scores of a warp's tile of slots against kRows query rows. Each thread has kKeys
// slots and kQ rows: key(i) within the tile, row(j) within the rows.
//
// On the tensor cores (bf16, D a multiple of 32): 16 slots are the rows of a product,
// 8 query rows its columns. The order of the dimensions within a dot product is
// free: a thread's 16 bytes of a slot's key serve two products as they are, and the
// same 16 bytes of a query are its share of the other operand.
template <int NT, int CHUNKS>
struct MmaScores {
  static constexpr int kTile = 16, kRows = 8 * NT, kKeys = 2, kQ = 2 * NT;
  static constexpr int kD = 32 * CHUNKS;
  static constexpr int kPitch = kD * 2 + 64;  // bytes of a query row in shared memory
  uint4 k[2][CHUNKS];

  __device__ static size_t smem_bytes(int) { return kRows * kPitch; }
  __device__ __forceinline__ static int key(int i) { return ((threadIdx.x & 31) >> 2) + 8 * i; }
  __device__ __forceinline__ static int row(int j) { return (j >> 1) * 8 + 2 * (threadIdx.x & 3) + (j & 1); }
  // lanes that share a row's columns differ in their upper three bits
  static constexpr int kFirstLane = 4;

  __device__ static void put_rows(const WeightParams& p, const unsigned char* q, int r0, int n, unsigned char* smem) {
    for (int i = threadIdx.x; i < kRows * (kD / 8); i += kWThreads) {
      const int r = i / (kD / 8), c = i % (kD / 8);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < n) {
        const int64_t t = (r0 + r) / p.G, g = (r0 + r) % p.G;
        v = load_unit(q + (t * p.q_token + g * p.q_head) * 2 + c * 16);
      }
      *reinterpret_cast<uint4*>(smem + r * kPitch + c * 16) = v;
    }
  }
  __device__ __forceinline__ void load(const WeightParams& p, const unsigned char* keys, int64_t first, int64_t end) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t s = first + key(i);
      const unsigned char* at = keys + s * p.k_slot * 2 + t * 16;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        k[i][c] = s < end ? __ldcs(reinterpret_cast<const uint4*>(at + c * 64)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void scores(const WeightParams&, const unsigned char* smem, float (&x)[kKeys][kQ]) const {
    const unsigned char* at = smem + ((threadIdx.x & 31) >> 2) * kPitch + (threadIdx.x & 3) * 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // (few columns: several chains of products, each waits for its last one)
      constexpr int kChains = NT == 1 ? 4 : NT == 2 ? 2 : 1;
      float cs[kChains][4] = {};
#pragma unroll
      for (int i = 0; i < CHUNKS; ++i) {
        const uint4 b = *reinterpret_cast<const uint4*>(at + n * 8 * kPitch + i * 64);
        const uint32_t a0[4] = {k[0][i].x, k[1][i].x, k[0][i].y, k[1][i].y};
        const uint32_t a1[4] = {k[0][i].z, k[1][i].z, k[0][i].w, k[1][i].w};
        mma_bf16(cs[2 * i % kChains], a0, b.x, b.y);
        mma_bf16(cs[(2 * i + 1) % kChains], a1, b.z, b.w);
      }
      float(&c)[4] = cs[0];
#pragma unroll
      for (int j = 1; j < kChains; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] += cs[j][i];
      x[0][2 * n] = c[0];
      x[0][2 * n + 1] = c[1];
      x[1][2 * n] = c[2];
      x[1][2 * n + 1] = c[3];
    }
  }
};

// In fp32, of any type and size: a slot a lane, ROWS query rows that the warp
// reads together.
template <int DT, int ROWS>
struct FmaScores {
  static constexpr int kTile = 32, kRows = ROWS, kKeys = 1, kQ = ROWS;
  static constexpr int kFirstLane = 1;
  const unsigned char* at;
  bool live;

  __device__ __forceinline__ static int key(int) { return threadIdx.x & 31; }
  __device__ __forceinline__ static int row(int j) { return j; }

  __device__ static void put_rows(const WeightParams& p, const unsigned char* q, int r0, int n, unsigned char* smem) {
    float* to = reinterpret_cast<float*>(smem);  // [D][kRows]
    for (int i = threadIdx.x; i < kRows * p.D; i += kWThreads) {
      const int r = i % kRows, d = i / kRows;
      const int64_t t = (r0 + r) / p.G, g = (r0 + r) % p.G;
      to[i] = r < n ? Elem<DT>::load(q, t * p.q_token + g * p.q_head + d) : 0.f;
    }
  }
  __device__ __forceinline__ void load(const WeightParams& p, const unsigned char* keys, int64_t first, int64_t end) {
    const int64_t s = first + key(0);
    live = s < end;
    at = keys + s * p.k_slot * Elem<DT>::kBytes;
  }
  __device__ __forceinline__ void scores(const WeightParams& p, const unsigned char* smem, float (&x)[kKeys][kQ]) const {
#pragma unroll
    for (int j = 0; j < kQ; ++j) x[0][j] = 0.f;
    if (!live) return;
    const float4* q = reinterpret_cast<const float4*>(smem);
    constexpr int U = Elem<DT>::kUnit;
    int d = 0;
    if ((reinterpret_cast<uintptr_t>(at) & 15u) == 0)
      for (; d + U <= p.D; d += U) {
        float2 v[U / 2];
        Elem<DT>::unpack(load_unit(at + d * Elem<DT>::kBytes), v);
#pragma unroll
        for (int i = 0; i < U / 2; ++i) {
          step(v[i].x, q + ROWS / 4 * (d + 2 * i), x[0]);
          step(v[i].y, q + ROWS / 4 * (d + 2 * i + 1), x[0]);
        }
      }
    for (; d < p.D; ++d) step(Elem<DT>::load(at, d), q + ROWS / 4 * d, x[0]);
  }
  __device__ __forceinline__ static void step(float k, const float4* q, float (&x)[kQ]) {
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i) {
      const float4 a = q[i];
      x[4 * i] = fmaf(k, a.x, x[4 * i]);
      x[4 * i + 1] = fmaf(k, a.y, x[4 * i + 1]);
      x[4 * i + 2] = fmaf(k, a.z, x[4 * i + 2]);
      x[4 * i + 3] = fmaf(k, a.w, x[4 * i + 3]);
    }
  }
};

// Scores are kept in natural units, and exponents are formed of their differences.
template <typename SC, int BYTES>
__global__ void __launch_bounds__(kWThreads, 2) weights_kernel(const WeightParams p) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t rank = cluster_rank(), C = p.c.B * p.c.H == 0 ? 1u : gridDim.x / static_cast<uint32_t>(p.c.B * p.c.H);
  const int64_t bh = cluster_id(), b = bh / p.c.H, h = bh % p.c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = p.G * p.T, chunks = (R + p.rows - 1) / p.rows;
  // dynamic: sums of a chunk's rows by warp, sums of all rows, query rows, scores
  RowSum* by_warp = reinterpret_cast<RowSum*>(dynamic);
  RowSum* sums = by_warp + kWWarps * kMaxRowsAtOnce;
  RowSum* merged = sums + 2 * ((R + 1) / 2);
  unsigned char* rows = reinterpret_cast<unsigned char*>(merged + 2 * ((R + 1) / 2));
  if (C > 1) cluster_arrive_relaxed();
  const int32_t n = length_of(p.c, b, p.c.S);
  const int64_t last = static_cast<int64_t>(p.c.seen != nullptr ? p.c.seen[b] : n) - p.T;  // the first query's position
  const int64_t per = (static_cast<int64_t>(n) + C - 1) / C;
  const int64_t share = (per + SC::kTile - 1) / SC::kTile * SC::kTile;
  const int64_t lo = min(static_cast<int64_t>(n), rank * share), hi = min(static_cast<int64_t>(n), lo + share);
  const unsigned char* q = static_cast<const unsigned char*>(p.query) + (b * p.q_batch + h * p.G * p.q_head) * BYTES;
  const unsigned char* keys = static_cast<const unsigned char*>(p.keys) + (b * p.k_batch + h * p.k_head) * BYTES;
  float* weights = p.c.weights + bh * p.c.S;
  const int32_t* positions = p.c.positions != nullptr ? p.c.positions + bh * p.c.S : nullptr;
  const bool stashed = p.stash > 0;
  float* stash = reinterpret_cast<float*>(rows + p.rows * (sizeof(float) * (p.D + 16)));
  auto position = [&](int64_t s) { return positions != nullptr ? positions[s] : static_cast<int32_t>(s); };
  // The last position that each of a chunk's rows sees (no row past the last sees any);
  // a slot outside the share has one that none sees.
  __shared__ int32_t sees[kMaxRowsAtOnce];
  constexpr int32_t kNone = INT32_MAX;
  auto set_rows = [&](int r0, int nr) {
    __syncthreads();
    SC::put_rows(p, q, r0, nr, rows);
    if (tid < SC::kRows) {
      const int64_t at = last + (r0 + tid) / p.G;
      sees[tid] = tid < nr && at >= INT32_MIN ? static_cast<int32_t>(min(at, static_cast<int64_t>(kNone) - 1)) : INT32_MIN;
    }
    __syncthreads();
  };

  for (int c = 0; c < chunks; ++c) {
    const int r0 = c * p.rows, nr = min(p.rows, R - r0);
    set_rows(r0, nr);
    RowSum run[SC::kQ];
    constexpr bool kHeld = SC::kQ <= 8;  // what this thread's rows see, in registers
    int32_t held[kHeld ? SC::kQ : 1];
#pragma unroll
    for (int j = 0; j < SC::kQ; ++j) {
      run[j] = {-INFINITY, 0.f};
      if (kHeld) held[j] = sees[SC::row(j)];
    }
    SC next;  // the tile whose keys are on their way
    next.load(p, keys, lo + warp * SC::kTile, hi);
    float* mine = stash + r0 * p.stash;
    const int len = static_cast<int>(hi - lo);
    for (int o = warp * SC::kTile; o < len; o += kWWarps * SC::kTile) {
      const SC sc = next;
      float x[SC::kKeys][SC::kQ];
      int32_t at[SC::kKeys];
#pragma unroll
      for (int i = 0; i < SC::kKeys; ++i) at[i] = o + SC::key(i) < len ? position(lo + o + SC::key(i)) : kNone;
      next.load(p, keys, lo + o + kWWarps * SC::kTile, hi);
      sc.scores(p, rows, x);
#pragma unroll
      for (int j = 0; j < SC::kQ; ++j) {
        const int r = SC::row(j);
        const int32_t see = kHeld ? held[kHeld ? j : 0] : sees[r];
        float top = run[j].m;
#pragma unroll
        for (int i = 0; i < SC::kKeys; ++i) {
          x[i][j] = at[i] <= see ? x[i][j] * p.scale : -INFINITY;
          top = fmaxf(top, x[i][j]);
          if (stashed && r < nr) mine[r * p.stash + o + SC::key(i)] = x[i][j];  // (a tile is whole there)
        }
        if (top > run[j].m) {
          run[j].s *= ex2((run[j].m - top) * kLog2e);
          run[j].m = top;
        }
#pragma unroll
        for (int i = 0; i < SC::kKeys; ++i)  // (a visible NaN, or one of +inf, makes the sum NaN)
          if (x[i][j] != -INFINITY) run[j].s += ex2((x[i][j] - run[j].m) * kLog2e);
      }
    }
#pragma unroll
    for (int j = 0; j < SC::kQ; ++j)
#pragma unroll
      for (int o = 16; o >= SC::kFirstLane; o >>= 1) {
        RowSum other;
        other.m = __shfl_xor_sync(kAll, run[j].m, o);
        other.s = __shfl_xor_sync(kAll, run[j].s, o);
        sum_add(run[j], other);
      }
    if (lane < SC::kFirstLane) {
#pragma unroll
      for (int j = 0; j < SC::kQ; ++j) by_warp[warp * kMaxRowsAtOnce + SC::row(j)] = run[j];
    }
    __syncthreads();
    if (tid < nr) {
      RowSum all = by_warp[tid];
      for (int w = 1; w < kWWarps; ++w) sum_add(all, by_warp[w * kMaxRowsAtOnce + tid]);
      sums[r0 + tid] = all;
    }
  }
  // the rows' sums over the cluster
  if (C > 1) cluster_wait();
  row_sync(C);
  for (int r = tid; r < R; r += kWThreads) {
    RowSum all = sums[r];
    if (C > 1) {
      all = {-INFINITY, 0.f};
      for (uint32_t c0 = 0; c0 < C; c0 += 4) {  // (four loads under way)
        unsigned long long v[4];
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) v[c] = ld_dsmem_sum(map_rank(smem_u32(&sums[r]), min(c0 + c, C - 1)));
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c)
          if (c0 + c < C)
            sum_add(all, {__uint_as_float(static_cast<uint32_t>(v[c])), __uint_as_float(static_cast<uint32_t>(v[c] >> 32))});
      }
    }
    // (a row that sees nothing, or logits of -inf alone, adds 0)
    merged[r] = {all.s == 0.f ? 0.f : all.m, all.s == 0.f ? 0.f : 1.f / all.s};
  }
  if (C > 1) cluster_arrive();  // (waited for at the end: the others read this CTA's sums)
  __syncthreads();
  if (stashed) {
    for (int64_t s = lo + tid; s < hi; s += kWThreads) {
      const int32_t at = position(s);
      float w = 0.f;
      const float* x = stash + static_cast<int>(s - lo);
      for (int t = 0, r = 0; t < p.T; ++t, r += p.G)
        if (at <= last + t)
          for (int g = 0; g < p.G; ++g)
            w += ex2((x[(r + g) * p.stash] - merged[r + g].m) * kLog2e) * merged[r + g].s;
      weights[s] = p.decay != 0.f ? fmaf(p.decay, weights[s], w) : w;
    }
  }
  for (int c = 0; !stashed && c < chunks; ++c) {
    const int r0 = c * p.rows, nr = min(p.rows, R - r0);
    set_rows(r0, nr);
    for (int64_t s0 = lo + warp * SC::kTile; s0 < hi; s0 += kWWarps * SC::kTile) {
      SC sc;
      float x[SC::kKeys][SC::kQ];
      sc.load(p, keys, s0, hi);
      sc.scores(p, rows, x);
#pragma unroll
      for (int i = 0; i < SC::kKeys; ++i) {
        const int64_t s = s0 + SC::key(i);
        const int32_t at = s < hi ? position(s) : kNone;
        float w = 0.f;
#pragma unroll
        for (int j = 0; j < SC::kQ; ++j) {
          const int r = SC::row(j);
          if (r < nr && at <= sees[r]) w += ex2((x[i][j] * p.scale - merged[r0 + r].m) * kLog2e) * merged[r0 + r].s;
        }
#pragma unroll
        for (int o = 1; o < SC::kFirstLane; o <<= 1) w += __shfl_xor_sync(kAll, w, o);
        const float keep = c == 0 ? p.decay : 1.f;
        if ((lane & (SC::kFirstLane - 1)) == 0 && s < hi) weights[s] = keep != 0.f ? fmaf(keep, weights[s], w) : w;
      }
    }
  }
  if (C > 1) cluster_wait();
}

template <typename SC, int BYTES>
cudaError_t launch_weights_of(const WeightParams& p, cudaStream_t st) {
  WeightParams q = p;
  q.rows = SC::kRows;
  const int64_t R = static_cast<int64_t>(p.G) * p.T, pairs = p.c.B * p.c.H;
  const size_t fixed = sizeof(RowSum) * (kWWarps * kMaxRowsAtOnce + 4 * ((R + 1) / 2)) + q.rows * (sizeof(float) * (p.D + 16));
  constexpr size_t kMost = 200 * 1024, kHalfSm = 110 * 1024;
  if (fixed > kMost) return cudaErrorInvalidValue;
  // shares of the slots: enough for the device, and of no more scores than fit (beside
  // another CTA's, if that can be)
  uint32_t C = 1;
  auto floats = [&](uint32_t c) {
    const int64_t per = (p.c.S + c - 1) / c, share = (per + SC::kTile - 1) / SC::kTile * SC::kTile;
    return share + (4 - share % 16 + 16) % 16;  // (4 modulo 16: a tile's stores meet no bank twice)
  };
  auto fits = [&](uint32_t c, size_t most) { return R <= kMaxRowsAtOnce && fixed + static_cast<size_t>(floats(c) * R) * 4 <= most; };
  while (C < kMaxRanks && pairs * 2 * C <= INT32_MAX && p.c.S / (2 * C) >= kWWarps * SC::kTile &&
         (pairs * 2 * C <= 2 * device_sms() || (R <= kMaxRowsAtOnce && !fits(C, kHalfSm))))
    C *= 2;
  q.stash = fits(C, kMost) ? static_cast<int32_t>(floats(C)) : 0;
  const size_t smem = fixed + static_cast<size_t>(q.stash * R) * 4;
  auto* fn = &weights_kernel<SC, BYTES>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(fn, kMost, done);
  if (e != cudaSuccess) return e;
  return launch(fn, static_cast<unsigned>(pairs * C), kWThreads, C, st, smem, q);
}

template <int DT, int BYTES>
cudaError_t launch_weights_fma(const WeightParams& p, cudaStream_t st) {
  if (static_cast<int64_t>(p.G) * p.T <= 8) return launch_weights_of<FmaScores<DT, 8>, BYTES>(p, st);
  return launch_weights_of<FmaScores<DT, 16>, BYTES>(p, st);
}

template <int CHUNKS>
cudaError_t launch_weights_mma(const WeightParams& p, cudaStream_t st) {
  const int64_t R = static_cast<int64_t>(p.G) * p.T;
  if (R <= 8) return launch_weights_of<MmaScores<1, CHUNKS>, 2>(p, st);
  if (R <= 16) return launch_weights_of<MmaScores<2, CHUNKS>, 2>(p, st);
  return launch_weights_of<MmaScores<4, CHUNKS>, 2>(p, st);
}

// ---------------------------------------------------------------------------
// Eviction: the kept slots of each (sequence, kv head), then their rows.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kFew = 2048;            // keys of a CTA in the boundary's first bin, where they fit
constexpr int kMaxShare = 48 * 1024;  // keys a CTA keeps in shared memory

// Selection of the first `keep` slots in order: the keep-th largest key by histograms
// of 11, 11 and 10 bits (integers: any order of the atomics gives the same), then the
// slots above it and the first of those equal to it, in slot order. The first digit has
// a weight's exponent and two bits more, so that few of a warp's weights meet in a bin;
// the last digit needs the keys alone that share it. A row has one CTA while its keys
// fit in shared memory: a barrier of a cluster costs as much as a thousand keys. Issue
// slots bound it: 128 rows of 32768 slots 25 us, of 1500 slots 5.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  uint32_t* own = reinterpret_cast<uint32_t*>(dynamic);
  __shared__ uint32_t few[kFew];
  __shared__ uint32_t n_few;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t all[kBins];
  __shared__ uint32_t counts[1];           // this CTA's protected slots
  __shared__ uint32_t above_of, digit_of;
  __shared__ uint32_t warp_more[kSelWarps], warp_same[kSelWarps];
  __shared__ uint32_t tally[2];            // this CTA's slots above the boundary, and equal to it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t rank = cluster_rank(), C = gridDim.x / static_cast<uint32_t>(p.c.B * p.c.H);
  const int64_t bh = cluster_id(), b = bh / p.c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t n = length_of(p.c, b, p.c.S);
  const int32_t keep = min(n, p.c.budget);
  const Guard guard(p.c, b, n);
  const float* weights = p.c.weights + bh * p.c.S;
  const int32_t* positions = p.c.positions != nullptr ? p.c.positions + bh * p.c.S : nullptr;
  int32_t* slots = p.out_slots + bh * p.c.budget;
  if (rank == 0) {
    if (bh % p.c.H == 0 && tid == 0) p.out_lengths[b] = keep;
    for (int64_t i = static_cast<int64_t>(keep) + tid; i < p.c.budget; i += kSelThreads) slots[i] = -1;
  }
  if (n <= p.c.budget) {  // (the same in every CTA of the cluster)
    for (int64_t i = rank * kSelThreads + tid; i < n; i += C * kSelThreads) slots[i] = static_cast<int32_t>(i);
    return;
  }
  if (C > 1) cluster_arrive_relaxed();  // every CTA of the cluster runs before its memory is read
  const int64_t share = (static_cast<int64_t>(n) + C - 1) / C;
  const int32_t lo = static_cast<int32_t>(min(static_cast<int64_t>(n), rank * share));
  const int32_t hi = static_cast<int32_t>(min(static_cast<int64_t>(n), lo + share));
  const bool kept_here = share <= p.share;
  auto raw = [&](int32_t s, bool& held) {
    held = guard.holds(positions != nullptr ? positions[s] : s);
    return weight_key(weights[s]);
  };
  if (tid == 0) counts[0] = n_few = 0u;
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0u;
  __syncthreads();
  // Protected slots: they are kept, or (more than the budget) the choice is theirs. The
  // keys go to shared memory and, while that is the usual case, to the first histogram.
  uint32_t mine = 0;
  auto take = [&](int64_t s, float w, int32_t at) {
    const bool held = guard.holds(at);
    const uint32_t k = held ? 0xFFFFFFFFu : weight_key(w);
    mine += held;
    atomicAdd(&hist[k >> 21], 1u);
    return k;
  };
  if (kept_here && ((reinterpret_cast<uintptr_t>(weights + lo) | reinterpret_cast<uintptr_t>(positions)) & 15u) == 0 &&
      (positions == nullptr || (reinterpret_cast<uintptr_t>(positions + lo) & 15u) == 0)) {
    constexpr int kFlight = 4;  // 16-byte loads of a thread under way
    const int n4 = (hi - lo) / 4;
    for (int i0 = tid; i0 < n4; i0 += kFlight * kSelThreads) {
      float4 w[kFlight];
      int4 at[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int j = i0 + i * kSelThreads;
        if (j >= n4) continue;
        w[i] = reinterpret_cast<const float4*>(weights + lo)[j];
        const int32_t s = lo + 4 * j;
        at[i] = positions != nullptr ? reinterpret_cast<const int4*>(positions + lo)[j] : make_int4(s, s + 1, s + 2, s + 3);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int j = i0 + i * kSelThreads;
        if (j >= n4) continue;
        const int64_t s = lo + 4 * j;
        uint4 k;
        k.x = take(s, w[i].x, at[i].x);
        k.y = take(s + 1, w[i].y, at[i].y);
        k.z = take(s + 2, w[i].z, at[i].z);
        k.w = take(s + 3, w[i].w, at[i].w);
        reinterpret_cast<uint4*>(own)[j] = k;
      }
    }
    const int32_t s = lo + 4 * n4 + tid;
    if (s < hi) own[s - lo] = take(s, weights[s], positions != nullptr ? positions[s] : s);
  } else {
    for (int64_t s = lo + tid; s < hi; s += kSelThreads) {
      const uint32_t k = take(s, weights[s], positions != nullptr ? positions[s] : static_cast<int32_t>(s));
      if (kept_here) own[s - lo] = k;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kAll, mine, o);
  if (lane == 0 && mine != 0u) atomicAdd(&counts[0], mine);
  if (C > 1) cluster_wait();
  row_sync(C);
  uint32_t held_all = 0;
  if (C == 1) held_all = counts[0];
  for (uint32_t c = 0; C > 1 && c < C; ++c) held_all += ld_dsmem_u32(map_rank(smem_u32(&counts[0]), c));
  const bool crowded = held_all > static_cast<uint32_t>(keep);
  // the key of slot s: of protected ones above all others, or all others below them
  auto made = [&](int32_t s) {
    bool held;
    const uint32_t k = raw(s, held);
    return crowded ? (held ? max(k, 1u) : 0u) : (held ? 0xFFFFFFFFu : k);
  };
  if (crowded && kept_here)
    for (int64_t s = lo + tid; s < hi; s += kSelThreads) own[s - lo] = made(static_cast<int32_t>(s));
  auto key = [&](int32_t s) { return kept_here ? own[s - lo] : made(s); };
  uint32_t prefix = 0, left = static_cast<uint32_t>(keep);  // the boundary's digits so far; its rank among those that share them
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round < 2 ? 11 : 10;
    const bool done = round == 0 && !crowded;  // (by the first pass)
    if (!done) {
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0u;
      __syncthreads();
    }
    if (done) {
    } else if (round == 2 && n_few <= kFew) {
      for (uint32_t i = tid; i < n_few; i += kSelThreads)
        if (few[i] >> 10 == prefix) atomicAdd(&hist[few[i] & 1023u], 1u);
    } else {
      const int all_of = (hi - lo + 31) / 32 * 32;  // (warps in step, for their ballots)
#pragma unroll 4
      for (int i = tid; i < all_of; i += kSelThreads) {
        const uint32_t k = i < hi - lo ? key(lo + i) : 0u;
        const bool in = i < hi - lo && (round == 0 || k >> (shift + bits) == prefix);
        if (in) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
        const uint32_t which = __ballot_sync(kAll, in);
        if (round == 1 && which != 0u) {
          uint32_t at = 0u;
          if (lane == 0) at = atomicAdd(&n_few, static_cast<uint32_t>(__popc(which)));
          at = __shfl_sync(kAll, at, 0) + __popc(which & ((1u << lane) - 1u));
          if (in && at < kFew) few[at] = k;
        }
      }
    }
    row_sync(C);
    const uint32_t* sums = hist;
    if (C > 1) {
      for (int i = tid; i < kBins; i += kSelThreads) {
        uint32_t v = 0;
        for (uint32_t c = 0; c < C; ++c) v += ld_dsmem_u32(map_rank(smem_u32(&hist[i]), c));
        all[i] = v;
      }
      row_sync(C);  // (the histograms have been read)
      sums = all;
    }
    // two bins a thread, the largest first
    constexpr int kEach = kBins / kSelThreads;
    static_assert(kEach == 2, "two bins a thread");
    const int top = kBins - 1 - kEach * tid;
    const uint32_t v0 = sums[top], v1 = sums[top - 1];
    uint32_t upto = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) warp_more[warp] = upto;
    __syncthreads();
    const uint32_t ahead = lane < warp ? warp_more[lane] : 0u;
    const uint32_t before = __reduce_add_sync(kAll, ahead) + upto - (v0 + v1);
    if (before < left && left <= before + v0) {
      digit_of = static_cast<uint32_t>(top);
      above_of = before;
    } else if (before + v0 < left && left <= before + v0 + v1) {
      digit_of = static_cast<uint32_t>(top - 1);
      above_of = before + v0;
    }
    __syncthreads();
    prefix = prefix << bits | digit_of;
    left -= above_of;
  }
  // Slots above the boundary and equal to it. A warp has a range of its own, 32 slots a
  // step; a lane keeps the ballots of one step of 32, so that no key is read again
  // where a range is 1024 slots or fewer.
  const int64_t span = ((static_cast<int64_t>(hi) - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int64_t w_lo = min(static_cast<int64_t>(hi), lo + warp * span), w_hi = min(static_cast<int64_t>(hi), w_lo + span);
  uint32_t gt = 0u, eq = 0u;  // of the lane's step
  auto ballots = [&](int64_t from) {
    gt = eq = 0u;
    const int steps = static_cast<int>(min((w_hi - from + 31) / 32, static_cast<int64_t>(32)));
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
      const int64_t s = from + 32 * i + lane;
      const bool some = s < w_hi;
      const uint32_t k = some ? key(static_cast<int32_t>(s)) : 0u;
      const uint32_t g = __ballot_sync(kAll, some && k > prefix), e = __ballot_sync(kAll, some && k == prefix);
      if (lane == i) {
        gt = g;
        eq = e;
      }
    }
    return steps;
  };
  constexpr int kSpan = 32 * 32;
  uint32_t more = 0, same = 0;
  for (int64_t from = w_lo; from < w_hi; from += kSpan) {
    ballots(from);
    more += __reduce_add_sync(kAll, static_cast<uint32_t>(__popc(gt)));
    same += __reduce_add_sync(kAll, static_cast<uint32_t>(__popc(eq)));
  }
  if (lane == 0) {
    warp_more[warp] = more;
    warp_same[warp] = same;
  }
  __syncthreads();
  // those of the warps before this one, and of the CTAs before
  uint32_t m0 = __reduce_add_sync(kAll, lane < warp ? warp_more[lane] : 0u);
  uint32_t e0 = __reduce_add_sync(kAll, lane < warp ? warp_same[lane] : 0u);
  if (C > 1) {
    if (tid == kSelThreads - 1) {
      tally[0] = m0 + more;
      tally[1] = e0 + same;
    }
    cluster_sync_all();
    for (uint32_t c = 0; c < rank; ++c) {
      m0 += ld_dsmem_u32(map_rank(smem_u32(&tally[0]), c));
      e0 += ld_dsmem_u32(map_rank(smem_u32(&tally[1]), c));
    }
    cluster_arrive();
  }
  for (int64_t from = w_lo; from < w_hi; from += kSpan) {
    int steps = 32;
    if (span > kSpan)
      steps = ballots(from);
    else
      steps = static_cast<int>((w_hi - from + 31) / 32);
    uint32_t m = __popc(gt), e = __popc(eq);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t um = __shfl_up_sync(kAll, m, o), ue = __shfl_up_sync(kAll, e, o);
      if (lane >= o) {
        m += um;
        e += ue;
      }
    }
    const uint32_t e_before = e0 + e - __popc(eq), m_before = m0 + m - __popc(gt);
    // of the equal ones, those that there is room for
    uint32_t kept = eq;
    const uint32_t room = left > e_before ? left - e_before : 0u;
    while (static_cast<uint32_t>(__popc(kept)) > room) kept &= ~(0x80000000u >> __clz(kept));
    kept |= gt;
    const uint32_t first = m_before + min(e_before, left);
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
      const uint32_t mask = __shfl_sync(kAll, kept, i), at = __shfl_sync(kAll, first, i);
      if (mask >> lane & 1u) slots[at + __popc(mask & ((1u << lane) - 1u))] = static_cast<int32_t>(from) + 32 * i + lane;
    }
    m0 += __shfl_sync(kAll, m, 31);
    e0 += __shfl_sync(kAll, e, 31);
  }
  if (C > 1) cluster_wait();
}

// Copies a row of bytes by N threads, in units of 16, 4 or 1 bytes as both ends
// allow; from null writes zeros.
template <int UNIT>
struct UnitOf {
  using T = uint4;
};
template <>
struct UnitOf<4> {
  using T = uint32_t;
};
template <>
struct UnitOf<1> {
  using T = unsigned char;
};

constexpr int kGatherThreads = 256;

// Weights and positions of `count` kept slots from the first-th on; by N threads.
template <int N>
__device__ __forceinline__ void gather_order(const EvictParams& p, int64_t bh, int64_t first, int count) {
  for (int i = threadIdx.x; i < count; i += N) {
    const int32_t s = p.out_slots[bh * p.c.budget + first + i];
    float w = 0.f;
    int32_t at = -1;
    if (s >= 0) {
      w = p.c.weights[bh * p.c.S + s];
      at = p.c.positions != nullptr ? p.c.positions[bh * p.c.S + s] : s;
    }
    p.out_weights[bh * p.out_slots_of + first + i] = w;
    p.out_positions[bh * p.out_slots_of + first + i] = at;
  }
}

// The kept rows: threads take units of rows in turn, several loads in flight.
template <int UNIT>
__device__ __forceinline__ void gather_rows(const CacheRows& from, const CacheRows& to, const EvictParams& p, int64_t bh,
                                            int64_t first, int64_t count) {
  using T = typename UnitOf<UNIT>::T;
  constexpr int kFlight = 4;
  const int64_t b = bh / p.c.H, h = bh % p.c.H;
  const uint32_t units = static_cast<uint32_t>(from.bytes / UNIT), total = static_cast<uint32_t>(count) * units;
  const unsigned char* src = static_cast<const unsigned char*>(from.at) + b * from.batch + h * from.head;
  unsigned char* dst = static_cast<unsigned char*>(to.at) + b * to.batch + h * to.head;
  const int32_t* slots = p.out_slots + bh * p.c.budget;
  for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kFlight * kGatherThreads) {
    T v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const uint32_t i = i0 + k * kGatherThreads;
      v[k] = T{};
      const int32_t s = i < total ? slots[first + i / units] : -1;
      if (s >= 0) v[k] = __ldcs(reinterpret_cast<const T*>(src + s * from.slot + static_cast<int64_t>(i % units) * UNIT));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const uint32_t i = i0 + k * kGatherThreads;
      if (i < total) *reinterpret_cast<T*>(dst + (first + i / units) * to.slot + static_cast<int64_t>(i % units) * UNIT) = v[k];
    }
  }
}

__device__ __forceinline__ uint64_t alignment_of(const CacheRows& r) {
  return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(r.at)) | static_cast<uint64_t>(r.bytes | r.batch | r.head | r.slot);
}

constexpr int kGatherRows = 64;
constexpr int kBulkThreads = 64;         // and rows of a CTA, at most
constexpr int kBulkBytes = 16 * 1024;    // of its rows
constexpr uint64_t kBulkLimitNs = 10ull * 1000 * 1000 * 1000;

// The same for rows of 16-byte units on their boundaries (16 x 8 rows of 32768 slots of
// 256 bytes cut to 4096: 78 us, 6.9 TB/s; by plain loads 95), by bulk copies (TMA): a
// thread asks for a row each, and the rows leave together where they lie one after
// another. Thirteen CTAs on an SM have 208 KB on their way.
__global__ void __launch_bounds__(kBulkThreads) evict_bulk_kernel(const EvictParams p, int per) {
  __shared__ __align__(128) unsigned char rows[kBulkBytes];
  __shared__ __align__(8) uint64_t bar;
  const int tid = threadIdx.x;
  if (tid == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t parts = (static_cast<int64_t>(p.c.budget) + per - 1) / per;
  const int64_t bh = blockIdx.x / parts, first = blockIdx.x % parts * per, b = bh / p.c.H, h = bh % p.c.H;
  const int count = static_cast<int>(min(static_cast<int64_t>(per), p.c.budget - first));
  const CacheRows& from = blockIdx.y == 0 ? p.key : p.value;
  const CacheRows& to = blockIdx.y == 0 ? p.out_key : p.out_value;
  const uint32_t bytes = static_cast<uint32_t>(from.bytes);
  unsigned char* dst = static_cast<unsigned char*>(to.at) + b * to.batch + h * to.head + first * to.slot;
  const int32_t s = tid < count ? p.out_slots[bh * p.c.budget + first + tid] : -1;
  const int some = __syncthreads_count(s >= 0);  // the rest have no token
  if (some > 0) {
    if (tid == 0) mbar_expect_tx(smem_u32(&bar), some * bytes);
    __syncthreads();
    if (s >= 0)
      bulk_g2s(smem_u32(rows) + tid * bytes, static_cast<const unsigned char*>(from.at) + b * from.batch + h * from.head + s * from.slot,
               bytes, smem_u32(&bar));
    if (blockIdx.y == 0) gather_order<kBulkThreads>(p, bh, first, count);
    const bool landed = __syncthreads_and(!p.give_up && mbar_wait_bounded(smem_u32(&bar), 0, kBulkLimitNs));
    if (landed) {
      const bool together = to.slot == from.bytes;
      if (together ? tid == 0 : s >= 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + (together ? 0 : tid * to.slot)),
                     "r"(smem_u32(rows) + (together ? 0u : tid * bytes)), "r"(together ? some * bytes : bytes)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    } else {
      // copies that do not land (not expected on a healthy device): the rows by plain loads;
      // the copies end, or a limit does, before their memory is given up
      for (int r = 0; r < some; ++r) {
        const int32_t at = p.out_slots[bh * p.c.budget + first + r];
        const unsigned char* src = static_cast<const unsigned char*>(from.at) + b * from.batch + h * from.head + at * from.slot;
        for (uint32_t i = tid * 16u; i < bytes; i += kBulkThreads * 16u)
          *reinterpret_cast<uint4*>(dst + r * to.slot + i) = load_unit(src + i);
      }
      mbar_wait_bounded(smem_u32(&bar), 0, kBulkLimitNs);
    }
  }
  if (some == 0 && blockIdx.y == 0) gather_order<kBulkThreads>(p, bh, first, count);
  for (int r = some; r < count; ++r)
    for (uint32_t i = tid * 16u; i < bytes; i += kBulkThreads * 16u)
      *reinterpret_cast<uint4*>(dst + r * to.slot + i) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t parts = (static_cast<int64_t>(p.c.budget) + kGatherRows - 1) / kGatherRows;
  const int64_t bh = blockIdx.x / parts, first = blockIdx.x % parts * kGatherRows;
  const int64_t count = min(static_cast<int64_t>(kGatherRows), p.c.budget - first);
  const CacheRows& from = blockIdx.y == 0 ? p.key : p.value;
  const CacheRows& to = blockIdx.y == 0 ? p.out_key : p.out_value;
  if (blockIdx.y == 0) gather_order<kGatherThreads>(p, bh, first, static_cast<int>(count));
  const uint64_t a = alignment_of(from) | alignment_of(to);
  if ((a & 15u) == 0u)
    gather_rows<16>(from, to, p, bh, first, count);
  else if ((a & 3u) == 0u)
    gather_rows<4>(from, to, p, bh, first, count);
  else
    gather_rows<1>(from, to, p, bh, first, count);
}

// ---------------------------------------------------------------------------
// One token a sequence: behind the last slot, or over the one that is last in order.
// ---------------------------------------------------------------------------
constexpr int kInsThreads = 256;

template <int UNIT>
__device__ __forceinline__ void copy_row(const unsigned char* from, unsigned char* to, int64_t bytes) {
  using T = typename UnitOf<UNIT>::T;
  for (int64_t i = threadIdx.x; i < bytes / UNIT; i += kInsThreads)
    reinterpret_cast<T*>(to)[i] = reinterpret_cast<const T*>(from)[i];
}

__device__ __forceinline__ void put_row(const CacheRows& from, const CacheRows& to, int64_t b, int64_t h, int64_t slot) {
  const unsigned char* src = static_cast<const unsigned char*>(from.at) + b * from.batch + h * from.head;
  unsigned char* dst = static_cast<unsigned char*>(to.at) + b * to.batch + h * to.head + slot * to.slot;
  const uint64_t a = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | static_cast<uint64_t>(from.bytes);
  if ((a & 15u) == 0u)
    copy_row<16>(src, dst, from.bytes);
  else if ((a & 3u) == 0u)
    copy_row<4>(src, dst, from.bytes);
  else
    copy_row<1>(src, dst, from.bytes);
}

// A cluster takes a sequence, its heads in turn; the sequence's length goes up
// when every CTA has read it. Latency bounds it: 64 x 8 x 4096 slots 7.5 us, 1 x 8 x
// 1000 3.1; one CTA walks a head, so 1 x 8 x 65536 takes 47.
__global__ void __launch_bounds__(kInsThreads) insert_kernel(const InsertParams p) {
  __shared__ unsigned long long least[kInsThreads / 32];
  __shared__ int32_t chosen;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t rank = cluster_rank(), C = gridDim.x / static_cast<uint32_t>(p.c.B);
  const int64_t b = cluster_id();
  const int tid = threadIdx.x;
  const int32_t given = p.c.lengths[b], seen = p.c.seen[b];
  if (given < 0) {  // (the same in every CTA of the cluster)
    for (int64_t h = static_cast<int64_t>(rank) * kInsThreads + tid; h < p.c.H; h += static_cast<int64_t>(C) * kInsThreads)
      p.out_slots[b * p.c.H + h] = -1;
    return;
  }
  const int32_t n = length_of(p.c, b, p.c.budget);
  const Guard guard(p.c, b, n);
  for (int64_t h = rank; h < p.c.H; h += C) {
    const int64_t row = (b * p.c.H + h) * p.c.S;
    if (n < p.c.budget) {
      if (tid == 0) chosen = n;
    } else {
      unsigned long long low = ~0ull;
      constexpr int kFlight = 8;  // loads of a thread under way
      for (int64_t s0 = tid; s0 < n; s0 += kFlight * kInsThreads) {
        float w[kFlight];
        int32_t at[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int64_t s = s0 + i * kInsThreads;
          w[i] = s < n ? p.c.weights[row + s] : 0.f;
          at[i] = s < n ? p.c.positions[row + s] : 0;
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int64_t s = s0 + i * kInsThreads;
          const unsigned long long held = guard.holds(at[i]);
          const unsigned long long k = held << 63 | static_cast<unsigned long long>(weight_key(w[i])) << 31 |
                                       static_cast<unsigned long long>(0x7FFFFFFF - s);
          if (s < n) low = min(low, k);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) low = min(low, __shfl_xor_sync(kAll, low, o));
      if ((tid & 31) == 0) least[tid >> 5] = low;
      __syncthreads();
      if (tid == 0) {
        for (int w = 1; w < kInsThreads / 32; ++w) low = min(low, least[w]);
        chosen = 0x7FFFFFFF - static_cast<int32_t>(low & 0x7FFFFFFFull);
      }
    }
    __syncthreads();
    const int32_t s = chosen;
    put_row(p.new_key, p.key, b, h, s);
    put_row(p.new_value, p.value, b, h, s);
    if (tid == 0) {
      p.c.weights[row + s] = 0.f;
      p.c.positions[row + s] = seen;
      p.out_slots[b * p.c.H + h] = s;
    }
    __syncthreads();  // (the next head's slot)
  }
  if (C > 1) cluster_sync_all();
  if (rank == 0 && tid == 0) {
    p.c.lengths[b] = min(n + 1, p.c.budget);
    p.c.seen[b] = seen + 1;
  }
}

}  // namespace

int launch_cache_weights(const WeightParams& p, int dtype, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == QRITA_DTYPE_F32) return static_cast<int>(launch_weights_fma<QRITA_DTYPE_F32, 4>(p, st));
  // rows of 16-byte units on their boundaries, 32 dimensions at a time: the tensor cores
  const uint64_t a = static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p.query) | reinterpret_cast<uintptr_t>(p.keys)) |
                     2u * static_cast<uint64_t>(p.q_batch | p.q_token | p.q_head | p.k_batch | p.k_head | p.k_slot);
  if ((a & 15u) == 0u) {
    int result;
    if (static_cast<int64_t>(p.G) * p.T > kFewRows && launch_cache_window(p, stream, &result)) return result;
    switch (p.D) {
      case 32: return static_cast<int>(launch_weights_mma<1>(p, st));
      case 64: return static_cast<int>(launch_weights_mma<2>(p, st));
      case 96: return static_cast<int>(launch_weights_mma<3>(p, st));
      case 128: return static_cast<int>(launch_weights_mma<4>(p, st));
      case 192: return static_cast<int>(launch_weights_mma<6>(p, st));
      case 256: return static_cast<int>(launch_weights_mma<8>(p, st));
      default: break;
    }
  }
  return static_cast<int>(launch_weights_fma<QRITA_DTYPE_BF16, 2>(p, st));
}

int launch_cache_evict(const EvictParams& p, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t pairs = p.c.B * p.c.H;
  uint32_t C = 1;
  while (C < kMaxRanks && p.c.S > static_cast<int64_t>(C) * kMaxShare && pairs * 2 * C <= INT32_MAX) C *= 2;
  EvictParams q = p;
  const int64_t share = (p.c.S + C - 1) / C;
  q.share = share <= kMaxShare ? static_cast<int32_t>(share) : 0;
  const size_t smem = static_cast<size_t>(q.share) * 4;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(&evict_select_kernel, kMaxShare * 4, done);
  if (e != cudaSuccess) return static_cast<int>(e);
  e = launch(&evict_select_kernel, static_cast<unsigned>(pairs * C), kSelThreads, C, st, smem, q);
  if (e != cudaSuccess) return static_cast<int>(e);
  auto aligned = [](const CacheRows& r) {
    return ((reinterpret_cast<uintptr_t>(r.at) | static_cast<uint64_t>(r.bytes | r.batch | r.head | r.slot)) & 15u) == 0u &&
           r.bytes <= kBulkBytes;
  };
  const bool bulk = aligned(p.key) && aligned(p.value) && aligned(p.out_key) && aligned(p.out_value);
  const int64_t widest = p.key.bytes > p.value.bytes ? p.key.bytes : p.value.bytes;
  const int per = !bulk ? kGatherRows : widest * kBulkThreads <= kBulkBytes ? kBulkThreads : static_cast<int>(kBulkBytes / widest);
  const int64_t parts = (static_cast<int64_t>(p.c.budget) + per - 1) / per;
  if (pairs * parts > INT32_MAX) return static_cast<int>(cudaErrorInvalidConfiguration);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * parts), 2, 1);
  cfg.blockDim = dim3(bulk ? kBulkThreads : kGatherThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = bulk ? cudaLaunchKernelEx(&cfg, &evict_bulk_kernel, q, per) : cudaLaunchKernelEx(&cfg, &evict_gather_kernel, q);
  const cudaError_t last = cudaGetLastError();
  return static_cast<int>(e != cudaSuccess ? e : last);
}

int launch_cache_insert(const InsertParams& p, qrita_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint32_t C = 1;
  while (C < 8 && 2 * C <= p.c.H) C *= 2;
  return static_cast<int>(launch(&insert_kernel, static_cast<unsigned>(p.c.B * C), kInsThreads, C, st, size_t(0), p));
}

}  // namespace qrita
