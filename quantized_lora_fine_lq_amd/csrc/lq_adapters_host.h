// Host-side helpers of the entry points that take sets of adapters.
#pragma once

#include "lq_adapters.h"
#include "lq_host.h"

namespace lq {

// Validate a set of adapters against an [N, K] weight and turn it into the kernels' view.
int check_set(const lq_adapter_set* set, int64_t N, int64_t K, AdapterView* v);

inline int64_t sum_r8(const lq_adapter_set* set) {
  const lq_adapter& last = set->host[set->n - 1];
  return (int64_t)last.row8 + (last.r + 7) / 8 * 8;
}

inline bool any_odd_rank(const lq_adapter_set* set) {
  for (int32_t a = 0; a < set->n; ++a)
    if (set->host[a].r % 8) return true;
  return false;
}

inline bool valid_M(int64_t M) { return M >= 1 && M < (int64_t(1) << 31); }

// The dropout generator counts a tensor's elements up to 2^47.
inline bool drop_fits(int64_t M, int64_t K) { return K < (int64_t(1) << 47) / M; }

inline size_t route_bytes(int64_t M, int32_t n) { return (size_t)route_words(M, n) * sizeof(int32_t); }

inline int64_t ldb_of(int64_t n) { return (n + 63) / 64 * 64; }

inline size_t bytes16(size_t elems) { return align_up(elems * sizeof(uint16_t)); }

}  // namespace lq
