// kv_attention_tree.cu -- attention of a step's rows (drafted trees, or one token) over the
// bf16 paged caches.
//
// Mathematics.  Row i of request r sees the positions [start, context) and context + j for the
// bits j of its mask, as far as the block table maps them to a block of the pool:
//   o_i = sum_p w_p v_p / sum_p w_p,  w_p = 2^(c q_i . k_p - ref),  c = scale * log2(e),
// in one pass with a running maximum ref.
#include <cuda_bf16.h>

#include <cfloat>

#include "kv_tree.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct TreeArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  int64_t num_blocks;
  BlockDiv div;
  int32_t q_heads, kv_heads, head_dim, group;
  const int32_t* table;
  int32_t stride;
  const int32_t* q_start;
  const int32_t* span_start;
  const int32_t* context_len;
  const int64_t* tree_mask;
  int32_t num_reqs, num_rows, max_rows;
  float scale_log2;
  __nv_bfloat16* out;
  int32_t* err;
};

// A CTA per (row of a request, query head); a warp takes every fourth key, a lane 4 channels.
__global__ void __launch_bounds__(kThreads) attention_tree_kernel(TreeArgs a) {
  __shared__ float s_o[kWarps][128], s_l[kWarps], s_ref[kWarps];
  pdl_allow_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y / a.max_rows, i = blockIdx.y - r * a.max_rows, qh = blockIdx.x;
  const StepRows rows = step_rows(a.q_start, r, a.num_rows, a.max_rows);
  uint32_t err = rows.count < 0 ? KV_ERR_BAD_QSL : 0;
  if (i >= rows.count) {
    if (i == 0 && qh == 0 && threadIdx.x == 0) report(a.err, err);
    return;
  }
  const int64_t start = a.span_start != nullptr ? a.span_start[r] : 0, ctx = a.context_len[r];
  const int64_t reach = (int64_t)a.stride * a.div.size;
  int64_t end = ctx + rows.count, lo = start;
  if (start < 0 || ctx < start) {
    err |= KV_ERR_BAD_POSITION;
    end = lo = 0;
  }
  if (end > reach && end > lo) {
    err |= KV_ERR_BAD_POSITION;
    end = reach;
  }
  const int64_t row = (int64_t)rows.first + i;
  const uint64_t mask = a.tree_mask != nullptr ? (uint64_t)a.tree_mask[row] : ~0ull >> (63 - i);
  const int h = qh / a.group, D = a.head_dim;
  const bool mine = 4 * lane < D;
  float q[4] = {};
  auto load4 = [&](const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * lane);
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  };
  if (mine) load4(a.q + row * a.q_stride + (int64_t)qh * D, q);
  float o[4] = {}, l = 0.f, ref = -INFINITY;
  for (int64_t p = lo + warp; p < end; p += kWarps) {
    int64_t lb, off;
    a.div.divmod(p, lb, off);
    const int32_t b = a.table[(int64_t)r * a.stride + lb];
    if (b == kNull) continue;
    if (b < 0 || b >= a.num_blocks) {
      err |= KV_ERR_BAD_BLOCK;
      continue;
    }
    if (p >= ctx && !((mask >> (p - ctx)) & 1)) continue;
    const int64_t at = (((int64_t)b * a.div.size + off) * a.kv_heads + h) * D;
    float k[4] = {}, v[4] = {};
    if (mine) {
      load4(a.k_cache + at, k);
      load4(a.v_cache + at, v);
    }
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    s *= a.scale_log2;
    if (s == -INFINITY) continue;
    const float up = fmaxf(ref, s), f = exp2f(ref - up), w = exp2f(s - up);
    ref = up;
    l = l * f + w;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = o[c] * f + w * v[c];
  }
  report(a.err, err);
#pragma unroll
  for (int c = 0; c < 4; ++c) s_o[warp][4 * lane + c] = o[c];
  if (lane == 0) s_l[warp] = l, s_ref[warp] = ref;
  __syncthreads();
  if ((int)threadIdx.x >= D) return;
  float top = -INFINITY, sum = 0.f, y = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ref[w]);
  if (top > -INFINITY)
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(s_ref[w] - top);
      sum += f * s_l[w];
      y += f * s_o[w][threadIdx.x];
    }
  a.out[(row * a.q_heads + qh) * D + threadIdx.x] = __float2bfloat16_rn(sum == 0.f ? 0.f : y / sum);
}

int sizes(int32_t num_reqs, int32_t max_rows, int32_t num_q_heads, int32_t num_kv_heads,
          int32_t head_dim) {
  if (num_reqs < 0 || max_rows < 1 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_q_heads % num_kv_heads != 0 || max_rows > kTreeRows)
    return KV_EINVAL;
  if (num_reqs > KV_MAX_GATHER_REQS || num_q_heads > 4096 || num_q_heads / num_kv_heads > 64 ||
      head_dim > 128 || head_dim % 8 != 0)
    return KV_EUNSUPPORTED;
  return KV_OK;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int64_t kv_attention_tree_workspace(int32_t num_reqs, int32_t max_rows,
                                               int32_t num_q_heads, int32_t num_kv_heads,
                                               int32_t head_dim) {
  const int rc = sizes(num_reqs, max_rows, num_q_heads, num_kv_heads, head_dim);
  return rc != KV_OK ? rc : 0;
}

extern "C" int kv_attention_tree(const void* query, int64_t query_stride, const void* k_cache,
                                 const void* v_cache, int32_t layer, int32_t num_layers,
                                 int64_t num_blocks, int32_t block_size, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim,
                                 const int32_t* block_table, int32_t table_stride,
                                 const int32_t* q_start_loc, const int32_t* span_start,
                                 const int32_t* context_len, const int64_t* tree_mask,
                                 int32_t num_reqs, int32_t num_rows, int32_t max_rows,
                                 float scale, void* out, void* workspace, int64_t workspace_bytes,
                                 int32_t* d_err, kv_stream_t stream) {
  int rc = step_checks(num_reqs, num_rows, d_err);
  if (rc != KV_OK) return rc;
  if (num_layers < 1 || layer < 0 || layer >= num_layers || num_blocks < 1 || block_size <= 0 ||
      table_stride < 0 || workspace_bytes < 0 || !(scale > 0.f) || !(scale < INFINITY))
    return KV_EINVAL;
  rc = sizes(num_reqs, max_rows, num_q_heads, num_kv_heads, head_dim);
  if (rc != KV_OK) return rc;
  const int64_t row = (int64_t)num_q_heads * head_dim;
  if (query_stride < row) return KV_EINVAL;
  if (query_stride % 8 != 0) return KV_EUNSUPPORTED;
  if (num_reqs == 0 || num_rows == 0) return KV_OK;
  if (query == nullptr || out == nullptr || k_cache == nullptr || v_cache == nullptr ||
      q_start_loc == nullptr || context_len == nullptr || !aligned(query, 16) ||
      !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(q_start_loc, 4) || !aligned(span_start, 4) || !aligned(context_len, 4) ||
      !aligned(tree_mask, 8) || !aligned(block_table, 4))
    return KV_EINVAL;
  if (table_stride > 0 && block_table == nullptr) return KV_EINVAL;
  const int64_t need =
      kv_attention_tree_workspace(num_reqs, max_rows, num_q_heads, num_kv_heads, head_dim);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
    return KV_EINVAL;
  const int64_t plane = num_blocks * block_size * num_kv_heads * head_dim * 2;
  const char* const k_layer = static_cast<const char*>(k_cache) + layer * plane;
  const char* const v_layer = static_cast<const char*>(v_cache) + layer * plane;
  const int64_t out_bytes = num_rows * row * 2;
  const auto over_input = [&](const void* p, int64_t bytes) {
    return overlap(p, bytes, query, ((num_rows - 1) * query_stride + row) * 2) ||
           overlap(p, bytes, k_layer, plane) || overlap(p, bytes, v_layer, plane) ||
           overlap(p, bytes, block_table, (int64_t)num_reqs * table_stride * 4) ||
           overlap(p, bytes, q_start_loc, (int64_t)(num_reqs + 1) * 4) ||
           overlap(p, bytes, span_start, (int64_t)num_reqs * 4) ||
           overlap(p, bytes, context_len, (int64_t)num_reqs * 4) ||
           overlap(p, bytes, tree_mask, (int64_t)num_rows * 8);
  };
  if (over_input(out, out_bytes) || over_input(workspace, need) ||
      overlap(out, out_bytes, workspace, need))
    return KV_EINVAL;
  const TreeArgs a{static_cast<const __nv_bfloat16*>(query), query_stride,
                   reinterpret_cast<const __nv_bfloat16*>(k_layer),
                   reinterpret_cast<const __nv_bfloat16*>(v_layer), num_blocks,
                   BlockDiv::make(block_size), num_q_heads, num_kv_heads, head_dim,
                   num_q_heads / num_kv_heads, block_table, table_stride, q_start_loc, span_start,
                   context_len, tree_mask, num_reqs, num_rows, max_rows,
                   fminf(scale * 1.44269504088896340736f, FLT_MAX),
                   static_cast<__nv_bfloat16*>(out), d_err};
  if ((int64_t)num_reqs * max_rows > 65535) return KV_EUNSUPPORTED;
  return launch_pdl(attention_tree_kernel, dim3((unsigned)num_q_heads, (unsigned)(num_reqs * max_rows)),
                    kThreads, 0, stream, a);
}
