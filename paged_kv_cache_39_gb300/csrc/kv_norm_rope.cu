// kv_norm_rope.cu -- per-head RMS norm of queries and keys, rotation by
// position, and the write of the new K and V rows to their cache slots.
//
// Mathematics.  For a head row x of D channels with weights w
//   y_i = x_i * w_i / sqrt(mean(x^2) + eps)
// and for every rotated pair (a, b) of y with the position's (c, s):
//   a' = a c - b s,  b' = b c + a s.
// Everything is held in 32 bits from the bf16 input to the one rounding of the
// output.
//
// GPU shape.  8 channels (4 pairs) per lane, so a head is D / 8 lanes and the
// sum of squares is a shuffle reduction inside them; with half-split pairs a
// lane holds 4 consecutive channels of each half (two 8-byte loads), with
// interleaved pairs 8 consecutive ones (one 16-byte load), so no pair ever
// crosses lanes.  A warp takes kSteps x (32 / lanes per head) heads of ONE
// token: the position, the slot and the (cos, sin) row are read once for all
// of them, and every head's load is issued before the first is used.
#include <cuda_bf16.h>

#include "kv_common.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 128;

struct NormRopeArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const int64_t* positions;
  const float* cos_sin;
  int64_t max_position;
  int32_t rotary_dim;
  float eps;
  int32_t num_tokens, q_heads, kv_heads, head_dim;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;    // may be null
  __nv_bfloat16* k_cache;  // both caches or neither
  __nv_bfloat16* v_cache;
  int64_t layer_base;      // layer * num_blocks
  int64_t num_blocks;
  int32_t block_size;
  const int64_t* slots;
  int32_t* err;
  int32_t units;           // warps per token
};

// The 8 channels of a lane: pairs (x[i], x[4 + i]), i < 4.
struct Pairs {
  uint2 a, b;
};

__device__ __forceinline__ void unpack4(const uint2& u, float* f) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <bool kInterleaved>
__device__ __forceinline__ Pairs load_pairs(const __nv_bfloat16* row, int ca, int cb) {
  Pairs p;
  if (kInterleaved) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + ca);
    p.a = make_uint2(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.z, u.w, 0x5410));
    p.b = make_uint2(__byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x7632));
  } else {
    p.a = *reinterpret_cast<const uint2*>(row + ca);
    p.b = *reinterpret_cast<const uint2*>(row + cb);
  }
  return p;
}

template <bool kInterleaved>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* row, int ca, int cb, const Pairs& p) {
  if (kInterleaved) {
    *reinterpret_cast<uint4*>(row + ca) =
        make_uint4(__byte_perm(p.a.x, p.b.x, 0x5410), __byte_perm(p.a.x, p.b.x, 0x7632),
                   __byte_perm(p.a.y, p.b.y, 0x5410), __byte_perm(p.a.y, p.b.y, 0x7632));
  } else {
    *reinterpret_cast<uint2*>(row + ca) = p.a;
    *reinterpret_cast<uint2*>(row + cb) = p.b;
  }
}

// kLanes: lanes per head (8, 16, 32: head_dim / 8 rounded up to a power of two).
template <int kLanes, bool kInterleaved, int kSteps>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a) {
  pdl_allow_next();
  pdl_wait();
  constexpr int kHeads = 32 / kLanes;  // heads of a warp step
  const int lane = threadIdx.x & 31;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t t = unit / a.units;
  if (t >= a.num_tokens) return;
  const int head0 = (int)(unit - t * a.units) * (kSteps * kHeads) + lane / kLanes;
  const int l = lane % kLanes;
  const int D = a.head_dim, R = a.rotary_dim;
  const bool active = l * 8 < D;
  // this lane's channels: pairs (ca + i, cb + i), rotated by pair index 4 l + i
  const bool rot = l * 8 < R;
  int ca, cb;
  if (kInterleaved) {
    ca = cb = 8 * l;
  } else if (rot) {
    ca = 4 * l;
    cb = R / 2 + 4 * l;
  } else {  // channels that are not rotated: the two halves of [R, D)
    ca = R + 4 * l - R / 2;
    cb = ca + (D - R) / 2;
  }
  const int total = a.q_heads + 2 * a.kv_heads;

  Pairs x[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * kHeads;
    x[s].a = x[s].b = make_uint2(0, 0);
    if (!active || h >= total) continue;
    if (h < a.q_heads) {
      x[s] = load_pairs<kInterleaved>(a.q + t * a.q_stride + (int64_t)h * D, ca, cb);
    } else if (h < a.q_heads + a.kv_heads) {
      x[s] = load_pairs<kInterleaved>(a.k + t * a.k_stride + (int64_t)(h - a.q_heads) * D, ca, cb);
    } else if (a.v_cache != nullptr) {
      x[s] = load_pairs<kInterleaved>(
          a.v + t * a.v_stride + (int64_t)(h - a.q_heads - a.kv_heads) * D, ca, cb);
    }
  }
  uint32_t err = 0;
  const int64_t pos = a.positions[t];
  const bool pos_ok = pos >= 0 && pos < a.max_position;
  if (!pos_ok) err |= KV_ERR_BAD_POSITION;
  int64_t cache_row = -1;
  if (a.k_cache != nullptr) {
    const int64_t s = a.slots[t];
    if (s >= 0) {
      const int64_t b = s / a.block_size;
      if (b == kNull) err |= KV_ERR_NULL_WRITE;
      else if (b >= a.num_blocks) err |= KV_ERR_BAD_SLOT;
      else if (pos_ok) cache_row = (a.layer_base + b) * a.block_size + (s - b * a.block_size);
    }
  }
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), z = make_float4(0.f, 0.f, 0.f, 0.f);
  if (rot && pos_ok) {
    const float* row = a.cos_sin + pos * R;
    c = *reinterpret_cast<const float4*>(row + 4 * l);
    z = *reinterpret_cast<const float4*>(row + R / 2 + 4 * l);
  }
  Pairs wq, wk;
  wq.a = wq.b = wk.a = wk.b = make_uint2(0, 0);
  if (active) {
    wq = load_pairs<kInterleaved>(a.q_weight, ca, cb);
    wk = load_pairs<kInterleaved>(a.k_weight, ca, cb);
  }
  const float inv_d = 1.0f / (float)D;
  const float cc[4] = {c.x, c.y, c.z, c.w}, zz[4] = {z.x, z.y, z.z, z.w};

#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * kHeads;
    const bool is_q = h < a.q_heads, is_k = !is_q && h < a.q_heads + a.kv_heads;
    float p[4], q[4], w[4], u[4];
    unpack4(x[s].a, p);
    unpack4(x[s].b, q);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += p[i] * p[i] + q[i] * q[i];
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
    const float r = rsqrtf(ss * inv_d + a.eps);
    unpack4(is_q ? wq.a : wk.a, w);
    unpack4(is_q ? wq.b : wk.b, u);
    float ya[4], yb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = p[i] * r * w[i], g = q[i] * r * u[i];
      ya[i] = rot ? f * cc[i] - g * zz[i] : f;
      yb[i] = rot ? g * cc[i] + f * zz[i] : g;
    }
    Pairs o;
    o.a = make_uint2(pack2(ya[0], ya[1]), pack2(ya[2], ya[3]));
    o.b = make_uint2(pack2(yb[0], yb[1]), pack2(yb[2], yb[3]));
    if (!pos_ok) o.a = o.b = make_uint2(0, 0);
    if (!active || h >= total) continue;
    if (is_q) {
      store_pairs<kInterleaved>(a.q_out + (t * a.q_heads + h) * D, ca, cb, o);
    } else if (is_k) {
      const int hk = h - a.q_heads;
      if (a.k_out != nullptr)
        store_pairs<kInterleaved>(a.k_out + (t * a.kv_heads + hk) * D, ca, cb, o);
      if (cache_row >= 0)
        store_pairs<kInterleaved>(a.k_cache + (cache_row * a.kv_heads + hk) * D, ca, cb, o);
    } else if (cache_row >= 0) {
      store_pairs<kInterleaved>(
          a.v_cache + (cache_row * a.kv_heads + h - a.q_heads - a.kv_heads) * D, ca, cb, x[s]);
    }
  }
  report(a.err, err);
}

template <int kLanes, bool kInterleaved>
int launch(NormRopeArgs a, cudaStream_t stream) {
  constexpr int kHeads = 32 / kLanes;
  const int heads = a.q_heads + a.kv_heads + (a.v_cache != nullptr ? a.kv_heads : 0);
  const int steps = (heads + kHeads - 1) / kHeads;
  constexpr int kSteps = 4;
  a.units = (steps + kSteps - 1) / kSteps;
  const int64_t warps = (int64_t)a.num_tokens * a.units;
  const int64_t ctas = (warps * 32 + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  return launch_pdl(norm_rope_kernel<kLanes, kInterleaved, kSteps>, (unsigned)ctas, kThreads, 0,
                    stream, a);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_qk_norm_rope_write(
    const void* query, int64_t query_stride, const void* key, int64_t key_stride,
    const void* value, int64_t value_stride, const void* q_weight, const void* k_weight,
    const int64_t* positions, const float* cos_sin, int64_t max_position, int32_t rotary_dim,
    int32_t interleaved, float eps, int32_t num_tokens, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, void* q_out, void* k_out, void* k_cache,
    void* v_cache, int32_t layer, int32_t num_layers, int64_t num_blocks, int32_t block_size,
    const int64_t* slot_mapping, int32_t* d_err, kv_stream_t stream) {
  const bool cached = k_cache != nullptr || v_cache != nullptr;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_position < 0 || rotary_dim <= 0 || rotary_dim > head_dim || !(eps >= 0.f))
    return KV_EINVAL;
  if (cached && (num_layers <= 0 || layer < 0 || layer >= num_layers || num_blocks < 1 ||
                 block_size <= 0))
    return KV_EINVAL;
  if (head_dim % 8 != 0 || head_dim > 256 || rotary_dim % 8 != 0) return KV_EUNSUPPORTED;
  if (num_q_heads > 65535 || num_kv_heads > 65535) return KV_EUNSUPPORTED;
  const int64_t q_row = (int64_t)num_q_heads * head_dim, k_row = (int64_t)num_kv_heads * head_dim;
  if (query_stride < q_row || key_stride < k_row || (cached && value_stride < k_row))
    return KV_EINVAL;
  if (query_stride % 8 != 0 || key_stride % 8 != 0 || (cached && value_stride % 8 != 0))
    return KV_EUNSUPPORTED;
  if (d_err != nullptr && !aligned(d_err, 4)) return KV_EINVAL;
  if (num_tokens == 0) return KV_OK;
  if (query == nullptr || key == nullptr || q_weight == nullptr || k_weight == nullptr ||
      positions == nullptr || q_out == nullptr || (cos_sin == nullptr && max_position > 0) ||
      (!cached && k_out == nullptr))
    return KV_EINVAL;
  if (cached && (k_cache == nullptr || v_cache == nullptr || value == nullptr ||
                 slot_mapping == nullptr))
    return KV_EINVAL;
  if (!aligned(query, 16) || !aligned(key, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(cos_sin, 16) ||
      !aligned(q_out, 16) || !aligned(k_out, 16))
    return KV_EINVAL;
  if (cached && (!aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
                 !aligned(slot_mapping, 8)))
    return KV_EINVAL;
  // In place is one head row per reader and writer; any other overlap of an
  // output with an input would let one warp write what another still reads.
  const int64_t n1 = num_tokens - 1;
  const int64_t q_bytes = (n1 * query_stride + q_row) * 2, k_bytes = (n1 * key_stride + k_row) * 2;
  const int64_t v_bytes = (n1 * value_stride + k_row) * 2;
  const int64_t qo = num_tokens * q_row * 2, ko = num_tokens * k_row * 2;
  const bool q_in_place = q_out == query && query_stride == q_row;
  const bool k_in_place = k_out == key && key_stride == k_row;
  if ((!q_in_place && overlap(q_out, qo, query, q_bytes)) || overlap(q_out, qo, key, k_bytes) ||
      (!k_in_place && overlap(k_out, ko, key, k_bytes)) || overlap(k_out, ko, query, q_bytes) ||
      overlap(q_out, qo, k_out, ko) ||
      (cached && (overlap(q_out, qo, value, v_bytes) || overlap(k_out, ko, value, v_bytes))))
    return KV_EINVAL;
  NormRopeArgs a{static_cast<const __nv_bfloat16*>(query),
                 static_cast<const __nv_bfloat16*>(key),
                 static_cast<const __nv_bfloat16*>(value),
                 query_stride, key_stride, value_stride,
                 static_cast<const __nv_bfloat16*>(q_weight),
                 static_cast<const __nv_bfloat16*>(k_weight),
                 positions, cos_sin, max_position, rotary_dim, eps, num_tokens, num_q_heads,
                 num_kv_heads, head_dim, static_cast<__nv_bfloat16*>(q_out),
                 static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(k_cache),
                 static_cast<__nv_bfloat16*>(v_cache),
                 cached ? (int64_t)layer * num_blocks : 0, num_blocks, block_size, slot_mapping,
                 d_err, 0};
  if (head_dim <= 64) return interleaved ? launch<8, true>(a, stream) : launch<8, false>(a, stream);
  if (head_dim <= 128)
    return interleaved ? launch<16, true>(a, stream) : launch<16, false>(a, stream);
  return interleaved ? launch<32, true>(a, stream) : launch<32, false>(a, stream);
}
