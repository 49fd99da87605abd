// C ABI of the key-value cache's entry points: argument checks. See include/qrita.h.

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <limits>

#include "qrita.h"
#include "qrita_cache.h"

namespace qrita {
namespace {

constexpr int64_t kMax = std::numeric_limits<int32_t>::max();
constexpr int64_t kMostRow = 1 << 20;    // bytes of a slot's key or value
constexpr int64_t kMostStride = int64_t(1) << 56;

bool stride_ok(int64_t s) { return s >= 0 && s <= kMostStride; }

// Sizes and [B, H, S] state; fills *out.
int order_args(int64_t B, int64_t H, int64_t S, float* weights, int32_t* positions, int32_t* lengths, int32_t* seen,
               int64_t most, CacheOrder* out) {
  // (products below 2^63, and every grid below 2^31 blocks)
  if (B < 0 || H < 1 || S < 1 || B > kMax || H > kMax || S > kMax) return QRITA_EINVAL;
  if (B > 0 && (B > most / H)) return QRITA_EUNSUPPORTED;
  out->B = B;
  out->H = H;
  out->S = S;
  out->weights = weights;
  out->positions = positions;
  out->lengths = lengths;
  out->seen = seen;
  out->budget = out->sink = out->recent = 0;
  if (B == 0) return QRITA_OK;
  if (weights == nullptr || lengths == nullptr || (positions == nullptr) != (seen == nullptr)) return QRITA_EINVAL;
  return QRITA_OK;
}

// Rows of `bytes` bytes: a pointer and three (two without slots) strides in bytes.
bool rows_ok(const void* at, int64_t bytes, const int64_t* strides, bool slots, CacheRows* out) {
  if (at == nullptr || strides == nullptr || bytes < 1 || bytes > kMostRow) return false;
  out->at = const_cast<void*>(at);
  out->bytes = bytes;
  out->batch = strides[0];
  out->head = strides[1];
  out->slot = slots ? strides[2] : 0;
  return stride_ok(out->batch) && stride_ok(out->head) && stride_ok(out->slot) && (!slots || out->slot >= bytes);
}

// Whether two caches' addresses overlap, from their first byte to their last.
bool overlap(const CacheRows& a, const CacheRows& b, int64_t B, int64_t H, int64_t slots_a, int64_t slots_b) {
  using Wide = unsigned __int128;
  auto end = [&](const CacheRows& r, int64_t slots) {
    return static_cast<Wide>(reinterpret_cast<uintptr_t>(r.at)) + static_cast<Wide>(r.batch) * (B - 1) +
           static_cast<Wide>(r.head) * (H - 1) + static_cast<Wide>(r.slot) * (slots - 1) + r.bytes;
  };
  return static_cast<Wide>(reinterpret_cast<uintptr_t>(a.at)) < end(b, slots_b) &&
         static_cast<Wide>(reinterpret_cast<uintptr_t>(b.at)) < end(a, slots_a);
}

// A contiguous vector's addresses.
struct Range {
  const void* at;  // null: there is none
  int64_t bytes;
};

bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x != 0 && y != 0 && x < y + static_cast<uint64_t>(b.bytes) && y < x + static_cast<uint64_t>(a.bytes);
}

// Whether a vector that is written overlaps another one, or one that is read. (A CTA
// writes its row's while others still read theirs: what they read would be a matter of
// timing.)
bool clash(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  for (const Range* w = written.begin(); w != written.end(); ++w) {
    for (const Range* v = written.begin(); v != w; ++v)
      if (overlap(*w, *v)) return true;
    for (const Range& r : read)
      if (overlap(*w, r)) return true;
  }
  return false;
}

bool budget_ok(int64_t S, int32_t budget, int32_t sink, int32_t recent, CacheOrder* out) {
  out->budget = budget;
  out->sink = sink;
  out->recent = recent;
  return budget >= 1 && budget <= kMax && sink >= 0 && recent >= 0 && S >= 1;
}

}  // namespace
}  // namespace qrita

extern "C" {

int qrita_cache_weights(int64_t B, int64_t H, int64_t S, const void* query, int dtype, int32_t T, int32_t G, int32_t D,
                        const int64_t* query_strides, const void* keys, const int64_t* key_strides, double scale,
                        double decay, const int32_t* lengths, const int32_t* positions, const int32_t* seen,
                        float* weights, qrita_stream_t stream) {
  return qrita_cache_weights_ex(B, H, S, query, dtype, T, G, D, query_strides, keys, key_strides, scale, decay, lengths,
                                positions, seen, weights, 0u, stream);
}

int qrita_cache_weights_ex(int64_t B, int64_t H, int64_t S, const void* query, int dtype, int32_t T, int32_t G, int32_t D,
                           const int64_t* query_strides, const void* keys, const int64_t* key_strides, double scale,
                           double decay, const int32_t* lengths, const int32_t* positions, const int32_t* seen,
                           float* weights, uint32_t flags, qrita_stream_t stream) {
  if ((flags & ~(QRITA_CACHE_FLAG_TEST_GIVE_UP_SUMS | QRITA_CACHE_FLAG_TEST_GIVE_UP_WEIGHTS)) != 0u) return QRITA_EINVAL;
  qrita::WeightParams prm = {};
  const int rc = qrita::order_args(B, H, S, weights, const_cast<int32_t*>(positions), const_cast<int32_t*>(lengths),
                                   const_cast<int32_t*>(seen), qrita::kMax / 16, &prm.c);
  if (rc != QRITA_OK) return rc;
  if (dtype != QRITA_DTYPE_F32 && dtype != QRITA_DTYPE_BF16) return QRITA_EINVAL;
  if (T < 1 || G < 1 || D < 1 || D > 1024 || static_cast<int64_t>(T) * G > 8192) return QRITA_EINVAL;
  if (!std::isfinite(static_cast<float>(scale)) || !(decay >= 0.0 && decay <= 1.0)) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (query == nullptr || keys == nullptr || query_strides == nullptr || key_strides == nullptr) return QRITA_EINVAL;
  const int64_t order = 4 * B * H * S;
  if (qrita::clash({{weights, order}}, {{lengths, 4 * B}, {positions, order}, {seen, 4 * B}})) return QRITA_EINVAL;
  const uint64_t eb = dtype == QRITA_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(query) % eb != 0 || reinterpret_cast<uintptr_t>(keys) % eb != 0) return QRITA_EINVAL;
  for (int i = 0; i < 3; ++i)
    if (!qrita::stride_ok(query_strides[i]) || !qrita::stride_ok(key_strides[i])) return QRITA_EINVAL;
  prm.query = query;
  prm.q_batch = query_strides[0];
  prm.q_token = query_strides[1];
  prm.q_head = query_strides[2];
  prm.keys = keys;
  prm.k_batch = key_strides[0];
  prm.k_head = key_strides[1];
  prm.k_slot = key_strides[2];
  prm.G = G;
  prm.T = T;
  prm.D = D;
  prm.flags = flags;
  prm.scale = static_cast<float>(scale);
  prm.decay = static_cast<float>(decay);
  return qrita::launch_cache_weights(prm, dtype, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_cache_evict(int64_t B, int64_t H, int64_t S, const int32_t* lengths, const float* weights,
                      const int32_t* positions, const int32_t* seen, int32_t budget, int32_t sink, int32_t recent,
                      const void* keys, int64_t key_bytes, const int64_t* key_strides, const void* values,
                      int64_t value_bytes, const int64_t* value_strides, void* out_keys, const int64_t* out_key_strides,
                      void* out_values, const int64_t* out_value_strides, int64_t out_S, float* out_weights,
                      int32_t* out_positions, int32_t* out_slots, int32_t* out_lengths, qrita_stream_t stream) {
  return qrita_cache_evict_ex(B, H, S, lengths, weights, positions, seen, budget, sink, recent, keys, key_bytes, key_strides,
                              values, value_bytes, value_strides, out_keys, out_key_strides, out_values, out_value_strides,
                              out_S, out_weights, out_positions, out_slots, out_lengths, 0u, stream);
}

int qrita_cache_evict_ex(int64_t B, int64_t H, int64_t S, const int32_t* lengths, const float* weights,
                         const int32_t* positions, const int32_t* seen, int32_t budget, int32_t sink, int32_t recent,
                         const void* keys, int64_t key_bytes, const int64_t* key_strides, const void* values,
                         int64_t value_bytes, const int64_t* value_strides, void* out_keys, const int64_t* out_key_strides,
                         void* out_values, const int64_t* out_value_strides, int64_t out_S, float* out_weights,
                         int32_t* out_positions, int32_t* out_slots, int32_t* out_lengths, uint32_t flags,
                         qrita_stream_t stream) {
  if ((flags & ~QRITA_CACHE_FLAG_TEST_GIVE_UP_ROWS) != 0u) return QRITA_EINVAL;
  qrita::EvictParams prm = {};
  prm.give_up = (flags & QRITA_CACHE_FLAG_TEST_GIVE_UP_ROWS) != 0u;
  const int rc = qrita::order_args(B, H, S, const_cast<float*>(weights), const_cast<int32_t*>(positions),
                                   const_cast<int32_t*>(lengths), const_cast<int32_t*>(seen), qrita::kMax / 16, &prm.c);
  if (rc != QRITA_OK) return rc;
  if (!qrita::budget_ok(S, budget, sink, recent, &prm.c) || budget > out_S || out_S > qrita::kMax) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (!qrita::rows_ok(keys, key_bytes, key_strides, true, &prm.key) ||
      !qrita::rows_ok(values, value_bytes, value_strides, true, &prm.value) ||
      !qrita::rows_ok(out_keys, key_bytes, out_key_strides, true, &prm.out_key) ||
      !qrita::rows_ok(out_values, value_bytes, out_value_strides, true, &prm.out_value))
    return QRITA_EINVAL;
  for (const qrita::CacheRows* to : {&prm.out_key, &prm.out_value})
    if (qrita::overlap(prm.key, *to, B, H, S, budget) || qrita::overlap(prm.value, *to, B, H, S, budget)) return QRITA_EINVAL;
  if (out_weights == nullptr || out_positions == nullptr || out_slots == nullptr || out_lengths == nullptr) return QRITA_EINVAL;
  const int64_t order = 4 * B * H * S, out_order = 4 * B * H * out_S;
  if (qrita::clash({{out_weights, out_order}, {out_positions, out_order}, {out_slots, 4 * B * H * budget}, {out_lengths, 4 * B}},
                   {{weights, order}, {positions, order}, {lengths, 4 * B}, {seen, 4 * B}}))
    return QRITA_EINVAL;
  if (B * H > qrita::kMax / ((static_cast<int64_t>(budget) + 63) / 64)) return QRITA_EUNSUPPORTED;
  prm.out_slots_of = out_S;
  prm.out_weights = out_weights;
  prm.out_positions = out_positions;
  prm.out_slots = out_slots;
  prm.out_lengths = out_lengths;
  return qrita::launch_cache_evict(prm, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

int qrita_cache_insert(int64_t B, int64_t H, int64_t S, int32_t* lengths, int32_t* seen, float* weights,
                       int32_t* positions, int32_t budget, int32_t sink, int32_t recent, void* keys, int64_t key_bytes,
                       const int64_t* key_strides, void* values, int64_t value_bytes, const int64_t* value_strides,
                       const void* new_keys, const int64_t* new_key_strides, const void* new_values,
                       const int64_t* new_value_strides, int32_t* out_slots, qrita_stream_t stream) {
  qrita::InsertParams prm = {};
  const int rc = qrita::order_args(B, H, S, weights, positions, lengths, seen, qrita::kMax / 16, &prm.c);
  if (rc != QRITA_OK) return rc;
  if (!qrita::budget_ok(S, budget, sink, recent, &prm.c) || budget > S) return QRITA_EINVAL;
  if (B == 0) return QRITA_OK;
  if (positions == nullptr || out_slots == nullptr) return QRITA_EINVAL;
  if (!qrita::rows_ok(keys, key_bytes, key_strides, true, &prm.key) ||
      !qrita::rows_ok(values, value_bytes, value_strides, true, &prm.value) ||
      !qrita::rows_ok(new_keys, key_bytes, new_key_strides, false, &prm.new_key) ||
      !qrita::rows_ok(new_values, value_bytes, new_value_strides, false, &prm.new_value))
    return QRITA_EINVAL;
  const int64_t order = 4 * B * H * S;
  if (qrita::clash({{weights, order}, {positions, order}, {lengths, 4 * B}, {seen, 4 * B}, {out_slots, 4 * B * H}}, {}))
    return QRITA_EINVAL;
  prm.out_slots = out_slots;
  return qrita::launch_cache_insert(prm, stream) == 0 ? QRITA_OK : QRITA_ECUDA;
}

}  // extern "C"
