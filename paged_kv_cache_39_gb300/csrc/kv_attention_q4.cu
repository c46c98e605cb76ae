// kv_attention_q4.cu -- attention of one query token per request over the 4-bit
// paged cache.
//
// Mathematics.  Request r attends the positions [start, end) that its block
// table maps to a block of the pool; with k, v the values the 4-bit rows stand
// for (kv_q4.cuh)
//   o = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale q . k_p - max_p).
//
// Plain form: one warp per (request, query head), D / 32 channels per lane.
#include "kv_q4.cuh"

namespace kvp {
namespace {

struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  Q4Layout at;
  const int32_t* table;
  int32_t stride;
  const int32_t* start;
  const int32_t* end;
  int32_t num_reqs, q_heads;
  float scale;
  __nv_bfloat16* out;
  int32_t* err;
};

template <int G>
__global__ void __launch_bounds__(32) attention_q4_kernel(AttnArgs a) {
  pdl_allow_next();
  pdl_wait();
  constexpr int D = 32 * G;
  const int lane = threadIdx.x;
  const int r = blockIdx.x / a.q_heads, h = blockIdx.x % a.q_heads;
  const int hk = h / (a.q_heads / a.at.kv_heads);
  const int T = a.at.block_size;
  const int64_t s0 = a.start[r], s1 = a.end[r];
  uint32_t err = 0;
  const bool ok = s0 >= 0 && s1 >= s0;
  if (!ok) err |= KV_ERR_BAD_POSITION;
  float q[G], o[G], m = -INFINITY, l = 0.f;
  const int g = lane >> 2;
  for (int j = 0; j < G; ++j) {
    q[j] = __bfloat162float(a.q[r * a.q_stride + (int64_t)h * D + 32 * j + lane]);
    o[j] = 0.f;
  }
  for (int64_t p = s0; ok && p < s1; ++p) {
    const int64_t lb = p / T;
    if (lb >= a.stride) { err |= KV_ERR_BAD_POSITION; break; }
    const int64_t b = a.table[(int64_t)r * a.stride + lb];
    if (b == kNull) continue;
    if (b < 0 || b >= a.at.num_blocks) { err |= KV_ERR_BAD_BLOCK; continue; }
    const int64_t rec = a.at.record(b, hk);
    const int off = (int)(p - lb * T);
    auto val = [&](const uint8_t* c, int j) {
      const uint32_t byte = c[rec + a.at.codes(off) + 2 * G * g + 2 * j + ((lane >> 1) & 1)];
      const uint16_t sb = reinterpret_cast<const uint16_t*>(c + rec + a.at.scales(off))[j];
      return (float)((int)((lane & 1) ? byte >> 4 : byte & 15u) - 8) *
             __uint_as_float((uint32_t)sb << 16);
    };
    float s = 0.f;
    for (int j = 0; j < G; ++j) s += q[j] * val(a.k_cache, j);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    s *= a.scale;
    const float mn = fmaxf(m, s), f = m == mn ? 1.f : expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * f + w;
    for (int j = 0; j < G; ++j) o[j] = o[j] * f + w * val(a.v_cache, j);
  }
  for (int j = 0; j < G; ++j)
    a.out[((int64_t)r * a.q_heads + h) * D + 32 * j + lane] =
        __float2bfloat16_rn(l > 0.f || l != l ? o[j] / l : 0.f);
  report(a.err, err);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int64_t kv_attention_q4_workspace(int32_t num_reqs, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim) {
  if (num_reqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_q_heads % num_kv_heads != 0)
    return KV_EINVAL;
  return 0;
}

extern "C" int kv_attention_q4(const void* query, int64_t query_stride, const void* k_cache,
                               const void* v_cache, int32_t layer, int32_t num_layers,
                               int64_t num_blocks, int32_t block_size, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t head_dim,
                               const int32_t* block_table, int32_t table_stride,
                               const int32_t* span_start, const int32_t* span_end,
                               int32_t num_reqs, float scale, void* out, void* workspace,
                               int64_t workspace_bytes, int32_t* d_err, kv_stream_t stream) {
  const int rc = q4_checks(k_cache, v_cache, layer, num_layers, num_blocks, block_size,
                           num_kv_heads, head_dim, d_err);
  if (rc != KV_OK) return rc;
  if (num_reqs < 0 || table_stride < 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      !(scale > 0.f) || !(scale < INFINITY) || workspace_bytes < 0)
    return KV_EINVAL;
  if (num_reqs > KV_MAX_GATHER_REQS || num_q_heads > 4096) return KV_EUNSUPPORTED;
  if (query_stride < (int64_t)num_q_heads * head_dim) return KV_EINVAL;
  if (query_stride % 8 != 0) return KV_EUNSUPPORTED;
  if (num_reqs == 0) return KV_OK;
  if (query == nullptr || out == nullptr || span_start == nullptr || span_end == nullptr ||
      k_cache == nullptr || v_cache == nullptr || !aligned(query, 16) || !aligned(out, 16) ||
      !aligned(span_start, 4) || !aligned(span_end, 4))
    return KV_EINVAL;
  if (table_stride > 0 && (block_table == nullptr || !aligned(block_table, 4))) return KV_EINVAL;
  const int64_t row = (int64_t)num_q_heads * head_dim;
  if (overlap(out, num_reqs * row * 2, query, ((num_reqs - 1) * query_stride + row) * 2))
    return KV_EINVAL;
  const int64_t need = kv_attention_q4_workspace(num_reqs, num_q_heads, num_kv_heads, head_dim);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
    return KV_EINVAL;
  AttnArgs a{static_cast<const __nv_bfloat16*>(query), query_stride,
             static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
             Q4Layout{(int64_t)layer * num_blocks, num_blocks, block_size, num_kv_heads, head_dim},
             block_table, table_stride, span_start, span_end, num_reqs, num_q_heads, scale,
             static_cast<__nv_bfloat16*>(out), d_err};
  return launch_pdl(head_dim == 128 ? attention_q4_kernel<4> : attention_q4_kernel<2>,
                    (unsigned)((int64_t)num_reqs * num_q_heads), 32, 0, stream, a);
}
