// kv_tree_layout.cu -- masks and positions of drafted trees from their parents.
//
// Mathematics.  mask_i = 2^i + mask_parent(i), depth_i = bits of mask_i - 1.  Parents come
// before their children, so with up_i = parent(i) the steps
//   mask_i |= mask_up(i),  up_i = up_up(i)
// double the rows that are accounted for: 6 of them cover 64 rows.
//
// GPU shape.  A warp per request, two rows a lane, everything in registers and shuffles; the
// steps end when no row has anything above it that is not in its mask.  The call is launch and
// two dependent loads: 3.0 us for one tree of 8 rows, 3.4 for 256 trees of 1 to 64 rows (0.27 MB, 0.04 us
// of the memory's time).
#include "kv_tree.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 64;
constexpr int kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads)
tree_layout_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ q_start,
                   const int32_t* __restrict__ context_len, int32_t num_reqs, int32_t num_rows,
                   int64_t* __restrict__ tree_mask, int64_t* __restrict__ positions,
                   int64_t* __restrict__ cache_positions, int32_t* err_word) {
  pdl_allow_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= num_reqs) return;
  const StepRows rows = step_rows(q_start, r, num_rows, kTreeRows);
  const int64_t ctx = context_len[r];
  uint32_t err = 0;
  if (rows.count < 0) err |= KV_ERR_BAD_QSL;
  else if (rows.count > 0 && ctx < 0) err |= KV_ERR_BAD_POSITION;
  uint64_t mask[2];
  int up[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    mask[h] = 1ull << i;
    up[h] = -1;
    if (i > 0 && i < rows.count) {
      up[h] = parents != nullptr ? parents[rows.first + i] : i - 1;
      if (up[h] < 0 || up[h] >= i) {
        err |= KV_ERR_BAD_TREE;
        up[h] = -1;
      }
    }
  }
  while (__any_sync(kFull, up[0] >= 0 || up[1] >= 0)) {
    uint64_t above[2];
    int next[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int src = up[h] & 31;
      const uint64_t m0 = __shfl_sync(kFull, mask[0], src), m1 = __shfl_sync(kFull, mask[1], src);
      const int u0 = __shfl_sync(kFull, up[0], src), u1 = __shfl_sync(kFull, up[1], src);
      above[h] = up[h] < 0 ? 0 : up[h] < 32 ? m0 : m1;
      next[h] = up[h] < 0 ? -1 : up[h] < 32 ? u0 : u1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mask[h] |= above[h];
      up[h] = next[h];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i < rows.count) {
      const int64_t at = (int64_t)rows.first + i;
      tree_mask[at] = (int64_t)mask[h];
      positions[at] = ctx < 0 ? -1 : ctx + __popcll(mask[h]) - 1;
      cache_positions[at] = ctx < 0 ? -1 : ctx + i;
    }
  }
  report(err_word, err);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_tree_layout(const int32_t* parents, const int32_t* q_start_loc,
                              const int32_t* context_len, int32_t num_reqs, int32_t num_rows,
                              int64_t* tree_mask, int64_t* positions, int64_t* cache_positions,
                              int32_t* d_err, kv_stream_t stream) {
  const int rc = step_checks(num_reqs, num_rows, d_err);
  if (rc != KV_OK) return rc;
  if (num_reqs == 0 || num_rows == 0) return KV_OK;
  if (q_start_loc == nullptr || context_len == nullptr || tree_mask == nullptr ||
      positions == nullptr || cache_positions == nullptr || !aligned(parents, 4) ||
      !aligned(q_start_loc, 4) || !aligned(context_len, 4) || !aligned(tree_mask, 8) ||
      !aligned(positions, 8) || !aligned(cache_positions, 8))
    return KV_EINVAL;
  int64_t* const outs[3] = {tree_mask, positions, cache_positions};
  const int64_t bytes = (int64_t)num_rows * 8;
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], bytes, parents, (int64_t)num_rows * 4) ||
        overlap(outs[i], bytes, q_start_loc, (int64_t)(num_reqs + 1) * 4) ||
        overlap(outs[i], bytes, context_len, (int64_t)num_reqs * 4) ||
        overlap(outs[i], bytes, outs[(i + 1) % 3], bytes))
      return KV_EINVAL;
  }
  return launch_pdl(tree_layout_kernel, (num_reqs + kWarps - 1) / kWarps, kThreads, 0, stream,
                    parents, q_start_loc, context_len, num_reqs, num_rows, tree_mask, positions,
                    cache_positions, d_err);
}
