// kv_tree.cuh -- what the operators of a step with drafted rows share.
#pragma once

#include "kv_common.cuh"

namespace kvp {

constexpr int kTreeRows = KV_MAX_TREE_ROWS;

// A request's rows of the step; count < 0: out of order, out of range or too many.
struct StepRows {
  int32_t first, count;
};
__device__ __forceinline__ StepRows step_rows(const int32_t* q_start, int r, int32_t num_rows,
                                              int32_t most) {
  const int32_t a = q_start[r], b = q_start[r + 1];
  const bool ok = a >= 0 && b >= a && b <= num_rows && b - a <= most;
  return StepRows{a, ok ? b - a : -1};
}

// Counts of requests and rows that the four calls take.
inline int step_checks(int32_t num_reqs, int32_t num_rows, const int32_t* d_err) {
  if (num_reqs < 0 || num_rows < 0) return KV_EINVAL;
  if (num_reqs > KV_MAX_GATHER_REQS || num_rows > kTreeRows * KV_MAX_GATHER_REQS)
    return KV_EUNSUPPORTED;
  if (d_err != nullptr && !aligned(d_err, 4)) return KV_EINVAL;
  return KV_OK;
}

}  // namespace kvp
