// Attention weights of a window of queries: more than 16 rows (queries times the
// heads that share a kv head) at once, on the fifth-generation tensor cores.
//
// The formulas are those of qrita_cache.cu's weights_kernel. A cluster of CTAs takes
// a (sequence, kv head), a share of the slots each, in tiles of 128 slots. Scores are
// worked out twice, with the operands' roles changed, so that no sum crosses lanes:
//   first   Q K^T, a query row a lane of tensor memory: its thread keeps the row's
//           running maximum and sum over the slots;
//   second  K Q^T, a slot a lane: its thread adds up the slot's weights over the rows,
//           w = sum_r 2^(c (x_r - m_r)) / S_r, c = scale log2 e.
// Between them the rows' sums merge through distributed shared memory. Both products
// read the same tiles of shared memory (dimensions contiguous, swizzled over 128
// bytes). Keys are read again for the second product, last tiles first: what L2 still
// has.
//
// A CTA has an SM: four groups of four warps, the lanes' threads of a tile in turn,
// a warp that issues the products and one that asks for the tiles (TMA). Four
// accumulators of 128 columns, all of the tensor memory, and as many stages of keys as
// shared memory has, so that copies are under way while products and exponentials
// are. No other CTA of these kernels fits beside one, so none waits for columns that
// another holds.
//
// Keys bound it, read twice: 32 queries of 4 heads on 8 x 8 x 16384 slots of 128 bf16
// 98 us for 537 MB of tiles (5.5 TB/s; 453 MB of them from HBM, on 128 SMs), 16 queries
// 94; its exponentials are 69 us of their pipe. (mma.sync in blocks of 32 rows: 930 us.
// Keys by 16-byte copies of 64 threads, two CTAs an SM, two stages: 120. Two groups,
// columns loaded ahead of their use: 114. With exponents as c x less c m, one
// multiply-add, it took 96: wrong for large scores. From 97 then, an eighth of the
// exponentials by polynomials on the multiply-add pipe: 103, a quarter: 106.)
//
// A row's sum is taken by its lane's thread in each group: 32 columns are summed first,
// then added to the running sum, S / (128 C) additions of a thread for S slots on C CTAs
// (512 for 65536 slots on one), each off by half a unit of the sum.

#include <cfloat>
#include <cmath>
#include <cstring>
#include <cstddef>
#include <cstdint>

#include <cuda.h>

#include "qrita_cache.h"
#include "qrita_rows.cuh"

namespace qrita {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kLanes = 128;              // threads of a group, slots of a tile, rows at most
constexpr int kGroups = 4;
constexpr int kWindowThreads = kGroups * kLanes + 64;
constexpr int kBuffers = 4;              // accumulators
constexpr int kColumns = kBuffers * kLanes;
constexpr int kHalf = kLanes * 128;      // bytes of a tile's 64 dimensions
template <int HALVES>
constexpr int kStages = HALVES == 1 ? 8 : HALVES == 2 ? 5 : 2;
template <int HALVES>
constexpr int kWindowSmem = (1 + kStages<HALVES>) * HALVES * kHalf + 1024;
static_assert(kWindowSmem<1> > 114 * 1024, "one CTA on an SM");
constexpr uint64_t kWindowLimitNs = 10ull * 1000 * 1000 * 1000;

// Shared-memory operand: rows of 128 bytes, swizzled, eight rows 1024 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// bf16 operands with contiguous dimensions, fp32 accumulators, 128 rows, n columns.
__device__ __forceinline__ uint32_t product_shape(int n) {
  return 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(kLanes >> 4) << 24;
}

__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(shape), "r"(add ? 1u : 0u)
      : "memory");
}

// Arrives at bar when every product issued so far is done.
__device__ __forceinline__ void products_done(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A box of a tensor to shared memory, at bar.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// 32 columns of this lane, there after columns_wait.
__device__ __forceinline__ void columns32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

// (The words pass through, so that no use of them moves before the wait.)
__device__ __forceinline__ void columns_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Whether `yes` holds in all threads of a group.
__device__ __forceinline__ bool lanes_all(bool yes, int group) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %3, %2, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(yes ? 1u : 0u), "n"(kLanes), "r"(group + 1)
      : "memory");
  return r != 0u;
}

// A row's largest score and its sum of 2^(c (x - m)). (The difference comes first: c x
// by itself is rounded by 2^-24 of it, which for scores beyond 2^30 is more than an
// exponent.)
struct WindowSum {
  float m, s;
};

struct WindowParams {
  WeightParams w;
  int32_t rows, first;  // this launch's rows, and its first query
  int32_t queries;      // of a box of Q
};

template <int HALVES>
__global__ void __launch_bounds__(kWindowThreads, 1)
window_kernel(const WindowParams wp, const __grid_constant__ CUtensorMap query_map, const __grid_constant__ CUtensorMap key_map) {
  const WeightParams& p = wp.w;
  constexpr int kDepth = kStages<HALVES>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[kDepth], empty[kDepth], made[kBuffers], taken[kBuffers];
  __shared__ WindowSum sums[kGroups][kLanes];
  __shared__ float4 row_pairs[kLanes / 2];  // -m of two rows, 1 / S of the two
  __shared__ int tile_positions[kGroups][2][kLanes];
  __shared__ uint32_t tmem_at;
  __shared__ volatile int failed;  // a bounded wait gave up
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t q_at = base, k_at = base + HALVES * kHalf;
  if (tid == 0) {
    for (int i = 0; i < kDepth; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(smem_u32(&made[i]), 1);
      mbar_init(smem_u32(&taken[i]), kLanes);
    }
    fence_mbar_init();
    failed = 0;
  }
  // (tensor memory only after that: the kernel before may be about to take some)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kGroups * 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)),
                 "r"(static_cast<uint32_t>(kColumns))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    fence_before();
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  const uint32_t rank = cluster_rank(), C = gridDim.x / static_cast<uint32_t>(p.c.B * p.c.H);
  const int64_t bh = cluster_id(), b = bh / p.c.H, h = bh % p.c.H;
  const int32_t given = p.c.lengths[b];
  const int32_t n = static_cast<int32_t>(min(static_cast<int64_t>(max(given, 0)), p.c.S));
  // (the position of this launch's first query)
  const int64_t first = static_cast<int64_t>(p.c.seen != nullptr ? p.c.seen[b] : n) - p.T + wp.first;
  const int64_t per = (static_cast<int64_t>(n) + C - 1) / C;
  const int64_t share = (per + kLanes - 1) / kLanes * kLanes;
  const int64_t lo = min(static_cast<int64_t>(n), rank * share), hi = min(static_cast<int64_t>(n), lo + share);
  const int tiles = static_cast<int>((hi - lo + kLanes - 1) / kLanes);
  const int R = wp.rows, columns = (R + 15) / 16 * 16;
  const float scale = fminf(fabsf(p.scale) * kLog2e, FLT_MAX);  // (above 0: what is not seen stays -inf)
  // every CTA of the cluster runs before its memory is read (in a launch without
  // clusters, threads that arrive at the cluster's barrier ahead of others are held)
  if (C > 1) cluster_sync_all();
  // For the use-th completion (0, 1, ...). When a wait has given up (`quit`: at once) all
  // others do too, and nothing more is asked for or issued.
  auto wait = [&](uint64_t& bar, int use, bool quit = false) {
    const uint32_t at = smem_u32(&bar), phase = static_cast<uint32_t>(use) & 1u;
    if (!quit && failed == 0) {
      if (mbar_try_wait(at, phase)) return true;
      const uint64_t t0 = globaltimer_ns();
      for (uint32_t i = 1; failed == 0 && ((i & 63u) != 0u || globaltimer_ns() - t0 <= kWindowLimitNs); ++i)
        if (mbar_try_wait(at, phase)) return true;
    }
    failed = 1;
    return false;
  };
  // (tests: the first CTA of a sequence's first head, in its sums or in its weights)
  const uint32_t quits = rank == 0 && bh % p.c.H == 0 ? p.flags : 0u;
  int asked = 0;  // tiles that the copying thread has asked for, or whose products are issued

  if (warp == kGroups * 4 + 1) {
    // copies: Q once, then the tiles of keys, all of them twice; the second time last ones
    // first, which are the ones that L2 has
    if (C > 1) cluster_arrive();
    if (lane == 0) {
      for (int it = 0; it < 2 * tiles; ++it) {
        const int stage = it % kDepth;
        if (it >= kDepth && !wait(empty[stage], it / kDepth - 1)) break;
        const int s0 = static_cast<int>(lo) + (it < tiles ? it : 2 * tiles - 1 - it) * kLanes;
        const uint32_t to = k_at + stage * (HALVES * kHalf), bar = smem_u32(&full[stage]);
        const uint32_t q_bytes = it == 0 ? static_cast<uint32_t>(HALVES * 128 * wp.queries * p.G) : 0u;
        mbar_expect_tx(bar, HALVES * kHalf + q_bytes);
        if (it == 0) {
          for (int i = 0; i < HALVES; ++i)
            copy_box(q_at + i * kHalf, &query_map, i * 64, static_cast<int>(h) * p.G, wp.first, static_cast<int>(b), bar);
        }
        for (int i = 0; i < HALVES; ++i)
          copy_box(to + i * kHalf, &key_map, i * 64, s0, static_cast<int>(h), static_cast<int>(b), bar);
        asked = it + 1;
      }
    }
    __syncwarp();
    if (C > 1) {
      cluster_wait();
      cluster_arrive();
    }
  } else if (warp == kGroups * 4) {
    if (C > 1) cluster_arrive();
    // scores of a negative scale are those of -Q
    const uint32_t minus = p.scale < 0.f ? 1u : 0u;
    if (lane == 0) {
      for (int it = 0; it < 2 * tiles; ++it) {
        const int stage = it % kDepth, buf = it % kBuffers;
        if (!wait(full[stage], it / kDepth) || (it >= kBuffers && !wait(taken[buf], it / kBuffers - 1))) break;
        fence_after();
        const uint32_t k = k_at + stage * (HALVES * kHalf), d = tmem + buf * kLanes;
        const bool rows_first = it < tiles;
        const uint32_t shape = product_shape(rows_first ? kLanes : columns) | minus << (rows_first ? 13 : 14);
#pragma unroll
        for (int i = 0; i < HALVES * 4; ++i) {
          const uint32_t off = (i >> 2) * kHalf + (i & 3) * 32;
          const uint64_t qd = operand(q_at + off), kd = operand(k + off);
          product(d, rows_first ? qd : kd, rows_first ? kd : qd, shape, i > 0);
        }
        products_done(smem_u32(&empty[stage]));
        products_done(smem_u32(&made[buf]));
        asked = it + 1;
      }
    }
    __syncwarp();
    if (C > 1) {
      cluster_wait();
      cluster_arrive();
    }
  } else {
    const int group = warp >> 2, t = tid & (kLanes - 1);  // this thread's lane
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const int32_t* positions = p.c.positions != nullptr ? p.c.positions + bh * p.c.S : nullptr;
    float* weights = p.c.weights + bh * p.c.S;
    auto position = [&](int64_t s) {  // of a slot; one outside the share is seen by no query
      return s < lo || s >= hi ? INT32_MAX : positions != nullptr ? positions[s] : static_cast<int32_t>(s);
    };
    // (A wait that has given up ends no loop here: all lanes meet at every barrier. What
    // it leaves without its scores is NaN: a row's sum, with it every weight of a slot that
    // the row sees, or this CTA's weights, at the end.)
    // The rows' sums.
    bool summed = true;
    const int64_t see = first + t / p.G;  // the last position this thread's row sees
    float m = -FLT_MAX;                   // the largest score
    float2 s2 = both(0.f);
    int32_t at = position(lo + group * kLanes + t);
    int it = group;
    for (; it < tiles; it += kGroups) {
      int* of = tile_positions[group][(it / kGroups) & 1];
      of[t] = at;
      const bool all = lanes_all(at <= first, group);
      at = position(lo + static_cast<int64_t>(it + kGroups) * kLanes + t);
      summed = wait(made[it % kBuffers], it / kBuffers, (quits & QRITA_CACHE_FLAG_TEST_GIVE_UP_SUMS) != 0u && it == 0) && summed;
      __syncwarp();
      fence_after();
      const uint32_t from = mine + it % kBuffers * kLanes;
#pragma unroll 1
      for (int c = 0; c < kLanes; c += 32) {
        uint32_t words[32];
        columns32(from + c, words);
        columns_wait(words);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(words[i]);
        if (!all) {
          // (no exponential of what is not seen: its place is that of a logit of -inf)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (of[c + i] > see) x[i] = -INFINITY;
        }
        float most = x[0];
#pragma unroll
        for (int i = 1; i < 31; i += 2) most = fmax3(most, x[i], x[i + 1]);
        most = fmaxf(most, x[31]);
        if (most > m) {
          const float f = ex2((m - most) * scale);
          s2.x *= f;
          s2.y *= f;
          m = most;
        }
        const float2 cc = both(scale), nm = both(-m);
        float2 part = both(0.f);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 y = mul2(add2(make_float2(x[i], x[i + 1]), nm), cc);
          part = add2(part, make_float2(ex2(y.x), ex2(y.y)));
        }
        s2 = add2(s2, part);
      }
      fence_before();
      arrive(smem_u32(&taken[it % kBuffers]));
    }
    sums[group][t] = {m, summed ? s2.x + s2.y : NAN};
    auto all_groups = [&]() { asm volatile("bar.sync 15, %0;" ::"n"(kGroups * kLanes) : "memory"); };
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      all_groups();
    }
    if (group == 0) {
      WindowSum all = {-FLT_MAX, 0.f};
      for (uint32_t c = 0; c < C; ++c) {
        float o[kGroups], s[kGroups];  // (all under way at once)
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const uint32_t at = smem_u32(&sums[i][t]), from = C > 1 ? map_rank(at, c) : at;
          o[i] = ld_dsmem_f32(from);
          s[i] = ld_dsmem_f32(from + 4);
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const float most = fmaxf(all.m, o[i]);
          all.s = all.s * ex2((all.m - most) * scale) + s[i] * ex2((o[i] - most) * scale);
          all.m = most;
        }
      }
      // rows that see nothing, or scores of -inf alone, add 0; so do those past the last
      float* to = reinterpret_cast<float*>(&row_pairs[t >> 1]) + (t & 1);
      const bool none = all.s == 0.f || t >= R;
      to[0] = none ? 0.f : -all.m;
      to[2] = none ? 0.f : 1.f / all.s;
    }
    if (C > 1) cluster_arrive();  // (the other CTAs may end)
    all_groups();
    // The slots' weights.
    it = tiles + (group + kGroups - tiles % kGroups) % kGroups;
    at = position(lo + static_cast<int64_t>(2 * tiles - 1 - it) * kLanes + t);
    for (; it < 2 * tiles; it += kGroups) {
      const int64_t s = lo + static_cast<int64_t>(2 * tiles - 1 - it) * kLanes + t;
      // rows from here on see this slot
      const int64_t after = at == INT32_MAX ? INT64_MAX : at - first;
      const int least = after <= 0 ? 0 : after >= R ? R : static_cast<int>(min(after * p.G, static_cast<int64_t>(R)));
      at = position(s - kGroups * kLanes);
      wait(made[it % kBuffers], it / kBuffers, (quits & QRITA_CACHE_FLAG_TEST_GIVE_UP_WEIGHTS) != 0u && it == tiles);
      __syncwarp();
      fence_after();
      const uint32_t from = mine + it % kBuffers * kLanes;
      const bool all_rows = __all_sync(kAll, least == 0);
      float2 w = both(0.f);
#pragma unroll 1
      for (int c = 0; c < columns; c += 32) {
        uint32_t words[32];
        columns32(from + c, words);
        columns_wait(words);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(words[i]);
        const float2 cc = both(scale);
        if (all_rows && c + 32 <= R) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 row = row_pairs[(c + i) >> 1];
            const float2 y = mul2(add2(make_float2(x[i], x[i + 1]), make_float2(row.x, row.y)), cc);
            w = fma2(make_float2(ex2(y.x), ex2(y.y)), make_float2(row.z, row.w), w);
          }
        } else {  // (columns past the last row hold anything)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 row = row_pairs[(c + i) >> 1];
            const float2 y = mul2(add2(make_float2(x[i], x[i + 1]), make_float2(row.x, row.y)), cc);
            if (c + i >= least && c + i < R) w.x = fmaf(ex2(y.x), row.z, w.x);
            if (c + i + 1 >= least && c + i + 1 < R) w.y = fmaf(ex2(y.y), row.w, w.y);
          }
        }
      }
      fence_before();
      arrive(smem_u32(&taken[it % kBuffers]));
      if (s < hi) weights[s] = p.decay != 0.f ? fmaf(p.decay, weights[s], w.x + w.y) : w.x + w.y;
    }
  }
  __syncthreads();
  if (failed != 0) {
    // copies and products in flight end (or a limit does) before their memory is given up
    if (lane == 0 && warp == kGroups * 4 + 1)
      for (int it = max(0, asked - kDepth); it < asked; ++it)
        mbar_wait_bounded(smem_u32(&full[it % kDepth]), static_cast<uint32_t>(it / kDepth) & 1u, kWindowLimitNs);
    if (lane == 0 && warp == kGroups * 4 && asked > 0)
      mbar_wait_bounded(smem_u32(&made[(asked - 1) % kBuffers]), static_cast<uint32_t>((asked - 1) / kBuffers) & 1u, kWindowLimitNs);
    for (int64_t s = lo + tid; s < hi; s += kWindowThreads) p.c.weights[bh * p.c.S + s] = NAN;
    __syncthreads();
  }
  if (warp == kGroups * 4) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kColumns))
                 : "memory");
  }
  if (C > 1) cluster_wait();
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder of tensor maps (null: there is none).
EncodeTiled encoder() {
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled fn = known.load(std::memory_order_relaxed);
  if (fn != nullptr) return fn;
  void* at = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  fn = reinterpret_cast<EncodeTiled>(at);
  known.store(fn, std::memory_order_relaxed);
  return fn;
}

// A map of bf16 boxes of 64 columns, swizzled over their 128 bytes, of a tensor of
// four dimensions; strides in elements. False: it cannot be one (a stride of 0 of more
// than one row, say).
bool make_map(CUtensorMap* map, const void* at, const int64_t (&dims)[4], const int64_t (&strides)[3], int rows, int more) {
  EncodeTiled encode = encoder();
  if (encode == nullptr) return false;
  cuuint64_t size[4], step[3];
  for (int i = 0; i < 4; ++i) size[i] = static_cast<cuuint64_t>(dims[i]);
  for (int i = 0; i < 3; ++i) {
    if (dims[i + 1] > 1 && strides[i] == 0) return false;
    step[i] = dims[i + 1] > 1 ? static_cast<cuuint64_t>(strides[i]) * 2 : static_cast<cuuint64_t>(dims[0] + 7) / 8 * 16;
  }
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(more), 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(at), size, step, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HALVES>
cudaError_t launch_window_of(const WeightParams& p, const CUtensorMap& query, const CUtensorMap& key, cudaStream_t st) {
  const int64_t pairs = p.c.B * p.c.H;
  constexpr size_t smem = kWindowSmem<HALVES>;
  auto* fn = &window_kernel<HALVES>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  // As many CTAs as are on the device at once, with two tiles each at least, and
  // clusters of 8 at most: 16 SMs are rarely free together (8 heads of 32768 slots, 512
  // rows in four launches: 8 CTAs a head 229 us, 16 CTAs 276; 64 heads of 16384, 128
  // rows, with two groups: 2 CTAs a head 114, 1 CTA 216, 4 CTAs 122).
  uint32_t C = 1;
  while (C < 8 && pairs * 2 * C <= device_sms() && p.c.S >= kLanes * 2 * static_cast<int64_t>(C)) C *= 2;
  // as many whole queries at a time as there are lanes for
  const int each = kLanes / p.G;
  for (int t = 0; t < p.T; t += each) {
    WindowParams q;
    q.w = p;
    q.first = t;
    q.rows = (p.T - t < each ? p.T - t : each) * p.G;
    q.queries = each;
    if (t > 0) q.w.decay = 1.f;
    e = launch(fn, static_cast<unsigned>(pairs * C), kWindowThreads, C, st, smem, q, query, key);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

bool launch_cache_window(const WeightParams& p, qrita_stream_t stream, int* result) {
  if (p.G > kLanes || p.D > 256 || p.c.B > INT32_MAX || p.c.S > INT32_MAX - 2 * kLanes) return false;
  // (scores of 0 whatever their products: no multiple of the products' differences)
  if (std::fabs(p.scale) < 1e-37f) return false;
  CUtensorMap query, key;
  if (!make_map(&query, p.query, {p.D, p.c.H * p.G, p.T, p.c.B}, {p.q_head, p.q_token, p.q_batch}, p.G, kLanes / p.G) ||
      !make_map(&key, p.keys, {p.D, p.c.S, p.c.H, p.c.B}, {p.k_slot, p.k_head, p.k_batch}, kLanes, 1))
    return false;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  *result = static_cast<int>(p.D <= 64    ? launch_window_of<1>(p, query, key, st)
                             : p.D <= 128 ? launch_window_of<2>(p, query, key, st)
                                          : launch_window_of<4>(p, query, key, st));
  return true;
}

}  // namespace qrita
