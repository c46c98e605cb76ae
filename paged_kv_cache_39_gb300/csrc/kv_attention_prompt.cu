// kv_attention_prompt.cu -- causal attention of packed sequences with grouped
// heads.
//
// Mathematics.  Request r holds query rows i < m and key rows j < n; row i sees
// the keys j <= i + n - m (the last query sees every key):
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - max_j)
// with a running maximum and sum over one pass of the keys.
//
// Plain form: one warp per (query row, head), D / 32 channels per lane.
#include <cuda_bf16.h>

#include "kv_common.cuh"

namespace kvp {
namespace {

struct PromptArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* q_start;
  const int32_t* k_start;
  int32_t num_reqs, nq, nk, q_heads, kv_heads, head_dim;
  float scale;
  __nv_bfloat16* out;
  int32_t* err;
};

__global__ void __launch_bounds__(128) prompt_kernel(PromptArgs a) {
  pdl_allow_next();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  uint32_t err = 0;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.num_reqs;
       r += (int64_t)gridDim.x * blockDim.x) {
    const int q0 = a.q_start[r], q1 = a.q_start[r + 1], k0 = a.k_start[r], k1 = a.k_start[r + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk) err |= KV_ERR_BAD_QSL;
  }
  report(a.err, err);
  const int64_t t = w / a.q_heads;
  const int h = (int)(w - t * a.q_heads);
  if (t >= a.nq) return;
  const int r = find_span(a.q_start, a.num_reqs, (int32_t)t);
  if (r < 0) return;
  const int q0 = a.q_start[r], q1 = a.q_start[r + 1], k0 = a.k_start[r], k1 = a.k_start[r + 1];
  if (q0 < 0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk || t >= q1) return;
  const int64_t seen = (t - q0) + (int64_t)(k1 - k0) - (q1 - q0) + 1;
  const int D = a.head_dim, hk = h / (a.q_heads / a.kv_heads);
  float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    q[i] = c < D ? __bfloat162float(a.q[t * a.q_stride + (int64_t)h * D + c]) : 0.f;
  }
  for (int64_t j = 0; j < seen; ++j) {
    const __nv_bfloat16* kr = a.k + (k0 + j) * a.k_stride + (int64_t)hk * D;
    const __nv_bfloat16* vr = a.v + (k0 + j) * a.v_stride + (int64_t)hk * D;
    float s = 0.f, v[4];
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c < D) s += q[i] * __bfloat162float(kr[c]);
      v[i] = c < D ? __bfloat162float(vr[c]) : 0.f;
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    s *= a.scale;
    const float mn = fmaxf(m, s), f = m == mn ? 1.f : expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < 4; ++i) o[i] = o[i] * f + p * v[i];
  }
  for (int i = 0; i < 4; ++i) {
    const int c = lane + 32 * i;
    if (c < D) a.out[(t * a.q_heads + h) * D + c] = __float2bfloat16_rn(seen > 0 ? o[i] / l : 0.f);
  }
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_attention_prompt(const void* query, int64_t query_stride, const void* key,
                                   int64_t key_stride, const void* value, int64_t value_stride,
                                   const int32_t* q_start_loc, const int32_t* k_start_loc,
                                   int32_t num_reqs, int32_t num_q_tokens, int32_t num_k_tokens,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   float scale, void* out, int32_t* d_err, kv_stream_t stream) {
  if (num_reqs < 0 || num_q_tokens < 0 || num_k_tokens < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || num_q_heads % num_kv_heads != 0 ||
      !(scale > 0.f) || !(scale < INFINITY))
    return KV_EINVAL;
  if (head_dim % 8 != 0 || head_dim > 128 || num_q_heads / num_kv_heads > 128 ||
      num_q_heads > 4096 || num_reqs > KV_MAX_GATHER_REQS)
    return KV_EUNSUPPORTED;
  const int64_t q_row = (int64_t)num_q_heads * head_dim, k_row = (int64_t)num_kv_heads * head_dim;
  if (query_stride < q_row || key_stride < k_row || value_stride < k_row) return KV_EINVAL;
  if (query_stride % 8 != 0 || key_stride % 8 != 0 || value_stride % 8 != 0)
    return KV_EUNSUPPORTED;
  if (d_err != nullptr && !aligned(d_err, 4)) return KV_EINVAL;
  if (num_reqs == 0 || num_q_tokens == 0) return KV_OK;
  if (query == nullptr || out == nullptr || q_start_loc == nullptr || k_start_loc == nullptr ||
      !aligned(query, 16) || !aligned(out, 16) || !aligned(q_start_loc, 4) ||
      !aligned(k_start_loc, 4) || !aligned(key, 16) || !aligned(value, 16))
    return KV_EINVAL;
  if (num_k_tokens > 0 && (key == nullptr || value == nullptr)) return KV_EINVAL;
  const int64_t out_bytes = num_q_tokens * q_row * 2, n1 = num_k_tokens - 1;
  if (overlap(out, out_bytes, query, ((num_q_tokens - 1) * query_stride + q_row) * 2) ||
      (num_k_tokens > 0 && (overlap(out, out_bytes, key, (n1 * key_stride + k_row) * 2) ||
                            overlap(out, out_bytes, value, (n1 * value_stride + k_row) * 2))))
    return KV_EINVAL;
  PromptArgs a{static_cast<const __nv_bfloat16*>(query), static_cast<const __nv_bfloat16*>(key),
               static_cast<const __nv_bfloat16*>(value), query_stride, key_stride, value_stride,
               q_start_loc, k_start_loc, num_reqs, num_q_tokens, num_k_tokens, num_q_heads,
               num_kv_heads, head_dim, scale, static_cast<__nv_bfloat16*>(out), d_err};
  const int64_t ctas = ((int64_t)num_q_tokens * num_q_heads + 3) / 4;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  return launch_pdl(prompt_kernel, (unsigned)ctas, 128, 0, stream, a);
}
