// kv_cache_keep_path.cu -- the kept rows' K and V to consecutive cache positions.
//
// Mathematics.  For i = 1 .. kept: row(context + i) = row(context + path_i), with path going
// up, so path_i >= i; rows with path_i = i stay.  Moving i in order is right in place: a place
// written before is context + i' with i' < i <= path_i, no source of a later step.
//
// GPU shape.  A thread takes 16 bytes of a row, of one layer's K or V, and moves them for every i
// in order, loads of kBatch rows (and kItems such places) ahead of their stores: no thread reads what
// another one writes.  CTAs are (request, share of the layers' vectors), as many as run at once; each
// finds its request's moved rows for itself, in three dependent loads.
//
// Measured: 128 requests' 322 moved rows of 32 layers (8 heads x 128, 84 MB) 19.1 us, 4.4 TB/s: launch
// and the dependent loads are 4 of it, the rest is rows of 2 KB scattered over the pool.  4 times the
// CTAs 34 us (each finds the rows again), half of them 23; one request's 4 layers 3.6 us.
#include "kv_tree.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 128;
constexpr int kItems = 4;   // vectors of a thread at a time
constexpr int kBatch = 2;   // and rows

struct KeepArgs {
  uint4* k_cache;
  uint4* v_cache;
  int32_t num_layers;
  int64_t num_blocks;
  BlockDiv div;
  int32_t row_vecs;
  const int32_t* table;
  int32_t stride;
  const int32_t* q_start;
  const int32_t* context_len;
  const int32_t* path;
  const int32_t* num_kept;
  int32_t num_rows, shares;
  int32_t* err;
};

__global__ void __launch_bounds__(kThreads) keep_path_kernel(KeepArgs a) {
  __shared__ int64_t s_src[kTreeRows], s_dst[kTreeRows];  // moved rows of a layer, in order
  __shared__ int s_count;
  pdl_allow_next();
  pdl_wait();
  const int r = blockIdx.x / a.shares, share = blockIdx.x - r * a.shares;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const StepRows rows = step_rows(a.q_start, r, a.num_rows, kTreeRows);
    const int64_t ctx = a.context_len[r];
    const int kept = a.num_kept[r];
    uint32_t err = 0;
    if (rows.count < 0) err = KV_ERR_BAD_QSL;
    else if (rows.count > 0 && (kept < 0 || kept >= rows.count)) err = KV_ERR_BAD_TREE;
    else if (rows.count > 0 && ctx < 0) err = KV_ERR_BAD_POSITION;
    int count = 0;
    if (err == 0 && rows.count > 0) {
      int64_t src[2], dst[2];
      bool moved[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        moved[h] = false;
        src[h] = dst[h] = 0;
        if (i > kept) continue;
        const int p = a.path[rows.first + i];
        const int before = i > 0 ? a.path[rows.first + i - 1] : -1;
        if (p <= before || p >= rows.count || (i == 0 && p != 0)) {
          err |= KV_ERR_BAD_TREE;
          continue;
        }
        moved[h] = p != i;
        if (!moved[h]) continue;
        auto slot = [&](int64_t pos) {
          int64_t lb, off;
          a.div.divmod(pos, lb, off);
          if (lb >= a.stride) {
            err |= KV_ERR_BAD_POSITION;
            return (int64_t)0;
          }
          const int32_t b = a.table[(int64_t)r * a.stride + lb];
          if (b == kNull) err |= KV_ERR_NULL_WRITE;
          else if (b < 0 || b >= a.num_blocks) err |= KV_ERR_BAD_BLOCK;
          return (int64_t)b * a.div.size + off;
        };
        src[h] = slot(ctx + p);
        dst[h] = slot(ctx + i);
      }
      if (!__any_sync(kFull, err != 0)) {
        const uint32_t m0 = __ballot_sync(kFull, moved[0]), m1 = __ballot_sync(kFull, moved[1]);
        const uint32_t below = (1u << lane) - 1u;
        if (moved[0]) {
          s_src[__popc(m0 & below)] = src[0];
          s_dst[__popc(m0 & below)] = dst[0];
        }
        if (moved[1]) {
          s_src[__popc(m0) + __popc(m1 & below)] = src[1];
          s_dst[__popc(m0) + __popc(m1 & below)] = dst[1];
        }
        count = __popc(m0) + __popc(m1);
      }
    }
    if (lane == 0) s_count = count;
    if (share == 0) report(a.err, err);
  }
  __syncthreads();
  const int count = s_count;
  if (count == 0) return;
  // items: (layer, K or V, vector of a row), this CTA's share of them: where its first one is, and from there
  // step by step (a 64-bit division an item took as long as the copy)
  const int per_layer = 2 * a.row_vecs;
  const int64_t items = (int64_t)per_layer * a.num_layers, step = (int64_t)a.shares * kThreads;
  const int64_t plane = a.num_blocks * a.div.size * a.row_vecs;  // vectors of a layer
  const int64_t first = (int64_t)share * kThreads + threadIdx.x;
  const int step_layers = (int)(step / per_layer), step_rest = (int)(step - (int64_t)step_layers * per_layer);
  int layer = (int)(first / per_layer), rest = (int)(first - (int64_t)layer * per_layer);
  for (int64_t it = first; it < items; it += kItems * step) {
    uint4* base[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      base[k] = layer >= a.num_layers
                    ? nullptr
                    : (rest >= a.row_vecs ? a.v_cache + rest - a.row_vecs : a.k_cache + rest) + layer * plane;
      layer += step_layers;
      rest += step_rest;
      if (rest >= per_layer) rest -= per_layer, ++layer;
    }
    for (int i = 0; i < count; i += kBatch) {
      uint4 x[kItems][kBatch];
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (base[k] != nullptr && i + b < count) x[k][b] = base[k][s_src[i + b] * a.row_vecs];
#pragma unroll
      for (int k = 0; k < kItems; ++k)
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (base[k] != nullptr && i + b < count) st_stream(base[k] + s_dst[i + b] * a.row_vecs, x[k][b]);
    }
  }
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_cache_keep_path(void* k_cache, void* v_cache, int32_t num_layers,
                                  int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                                  int32_t head_dim, const int32_t* block_table,
                                  int32_t table_stride, const int32_t* q_start_loc,
                                  const int32_t* context_len, const int32_t* path,
                                  const int32_t* num_kept, int32_t num_reqs, int32_t num_rows,
                                  int32_t* d_err, kv_stream_t stream) {
  const int rc = step_checks(num_reqs, num_rows, d_err);
  if (rc != KV_OK) return rc;
  if (num_layers < 1 || num_blocks < 1 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      table_stride < 0)
    return KV_EINVAL;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (row % 8 != 0 || row / 8 > INT32_MAX / 2) return KV_EUNSUPPORTED;
  if (num_reqs == 0 || num_rows == 0) return KV_OK;
  if (k_cache == nullptr || v_cache == nullptr || q_start_loc == nullptr || context_len == nullptr ||
      path == nullptr || num_kept == nullptr || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_table, 4) || !aligned(q_start_loc, 4) || !aligned(context_len, 4) ||
      !aligned(path, 4) || !aligned(num_kept, 4))
    return KV_EINVAL;
  if (table_stride > 0 && block_table == nullptr) return KV_EINVAL;
  const int64_t bytes = row * 2 * block_size * num_blocks * num_layers;
  void* const caches[2] = {k_cache, v_cache};
  for (void* c : caches) {
    if (overlap(c, bytes, block_table, (int64_t)num_reqs * table_stride * 4) ||
        overlap(c, bytes, q_start_loc, (int64_t)(num_reqs + 1) * 4) ||
        overlap(c, bytes, context_len, (int64_t)num_reqs * 4) ||
        overlap(c, bytes, path, (int64_t)num_rows * 4) ||
        overlap(c, bytes, num_kept, (int64_t)num_reqs * 4) || overlap(c, bytes, d_err, 4))
      return KV_EINVAL;
  }
  if (overlap(k_cache, bytes, v_cache, bytes)) return KV_EINVAL;
  const int64_t items = 2 * (row / 8) * num_layers;
  int64_t shares = (items + kThreads - 1) / kThreads;
  const int64_t cap = (int64_t)sm_count() * (2048 / kThreads);  // CTAs that run at once
  const int64_t most = cap / num_reqs > 0 ? cap / num_reqs : 1;
  if (shares > most) shares = most;
  KeepArgs a{static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), num_layers, num_blocks,
             BlockDiv::make(block_size), (int32_t)(row / 8), block_table, table_stride, q_start_loc,
             context_len, path, num_kept, num_rows, (int32_t)shares, d_err};
  return launch_pdl(keep_path_kernel, (unsigned)(num_reqs * shares), kThreads, 0, stream, a);
}
