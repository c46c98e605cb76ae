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
// Both at once: a' = r (x_a (w_a c) - x_b (w_b s)) with r = 1 / sqrt(..), and the products
// of weights and angles are one set for all heads of a token.
//
// GPU shape.  The bytes bound a large batch, the chain position -> (cos, sin) -> store a small
// one.  8 channels (4 pairs) per lane, so a head is D / 8 lanes and the sum of squares is a
// shuffle reduction inside them; with half-split pairs a lane holds 4 consecutive channels of
// each half (two 8-byte loads), with interleaved pairs 8 consecutive ones (one 16-byte load),
// so no pair ever crosses lanes.  A warp takes kSteps x (32 / lanes per head) heads of one kind
// (query, key or value) of ONE token: position, slot and angles are read once for all of them
// and every head's load is issued before the first is used.  fp32 in pairs (one instruction for
// two).  Measured (32 query and 8 KV heads of 128 channels): 8432 tokens 40 us (229 MB, 5.7 TB/s),
// 256 tokens 4.0 us a call.  9 CTAs an SM (56 registers; a few spilled
// words in some forms): with 8 (none) 42.8 us, with 10 (up to 23 words) 40.9; 2, 3 or 8 steps
// instead of 4: 47.8, 47.8, 50.0.
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
  BlockDiv div;
  const int64_t* slots;
  int32_t* err;
  int32_t units, q_units, kv_units;  // warps per token; of them for queries; for keys
};

// The 8 channels of a lane: pairs (x[i], x[4 + i]), i < 4.
struct Pairs {
  uint2 a, b;
};

// Two bf16 values as a pair of fp32.
__device__ __forceinline__ uint64_t unpack2(uint32_t u) {
  return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
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

// kLanes: lanes per head (8, 16, 32: head_dim / 8 rounded up to a power of two).  kAll: every
// channel is rotated.
template <int kLanes, bool kInterleaved, bool kAll, int kSteps>
__global__ void __launch_bounds__(kThreads, 9) norm_rope_kernel(NormRopeArgs a) {
  pdl_allow_next();
  pdl_wait();
  constexpr int kHeads = 32 / kLanes;        // heads of a warp step
  constexpr int kUnit = kSteps * kHeads;     // heads of a warp
  const int lane = threadIdx.x & 31;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t t = unit <= INT32_MAX ? (uint32_t)unit / (uint32_t)a.units : unit / a.units;
  if (t >= a.num_tokens) return;
  // which heads: query units, then key units, then value units
  int u = (int)(unit - t * a.units);
  const bool is_q = u < a.q_units;
  const bool is_k = !is_q && u < a.q_units + a.kv_units;
  u -= is_q ? 0 : is_k ? a.q_units : a.q_units + a.kv_units;
  const int heads = is_q ? a.q_heads : a.kv_heads;
  const int head0 = u * kUnit + lane / kLanes;
  const int l = lane % kLanes;
  const int D = a.head_dim, R = a.rotary_dim;
  const bool active = l * 8 < D;
  // this lane's channels: pairs (ca + i, cb + i), rotated by pair index 4 l + i
  const bool rot = kAll || l * 8 < R;
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
  const __nv_bfloat16* in = is_q   ? a.q + t * a.q_stride
                            : is_k ? a.k + t * a.k_stride
                                   : a.v + t * a.v_stride;
  Pairs x[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * kHeads;
    x[s].a = x[s].b = make_uint2(0, 0);
    if (active && h < heads) x[s] = load_pairs<kInterleaved>(in + h * D, ca, cb);
  }
  uint32_t err = 0;
  const int64_t pos = a.positions[t];
  const bool pos_ok = pos >= 0 && pos < a.max_position;
  if (!pos_ok) err |= KV_ERR_BAD_POSITION;
  int64_t cache_row = -1;
  if (!is_q && a.k_cache != nullptr) {
    const int64_t s = a.slots[t];
    if (s >= 0) {
      int64_t b, off;
      a.div.divmod(s, b, off);
      if (b == kNull) err |= KV_ERR_NULL_WRITE;
      else if (b >= a.num_blocks) err |= KV_ERR_BAD_SLOT;
      else if (pos_ok) cache_row = (a.layer_base + b) * a.block_size + off;
    }
  }
  if (!is_q && !is_k) {  // values: their bits, to the cache
    __nv_bfloat16* out = a.v_cache + cache_row * a.kv_heads * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = head0 + s * kHeads;
      if (active && h < heads && cache_row >= 0) store_pairs<kInterleaved>(out + h * D, ca, cb, x[s]);
    }
    return;  // errors are reported by the keys' units
  }
  // weights times angles: a' = r (x_a wc_a - x_b ws_b), b' = r (x_b wc_b + x_a ws_a)
  uint64_t wc_a[2] = {}, wc_b[2] = {}, ws_a[2] = {}, ws_b[2] = {};
  if (active) {
    const Pairs w = load_pairs<kInterleaved>(is_q ? a.q_weight : a.k_weight, ca, cb);
    const uint64_t wa[2] = {unpack2(w.a.x), unpack2(w.a.y)};
    const uint64_t wb[2] = {unpack2(w.b.x), unpack2(w.b.y)};
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), z = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rot && pos_ok) {
      const float* row = a.cos_sin + pos * R;
      c = *reinterpret_cast<const float4*>(row + 4 * l);
      z = *reinterpret_cast<const float4*>(row + R / 2 + 4 * l);
    }
    const uint64_t cc[2] = {pair(c.x, c.y), pair(c.z, c.w)}, zz[2] = {pair(z.x, z.y), pair(z.z, z.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wc_a[i] = mul2(wa[i], cc[i]);
      wc_b[i] = mul2(wb[i], cc[i]);
      ws_a[i] = mul2(wa[i], zz[i]);
      ws_b[i] = mul2(wb[i], zz[i]) ^ 0x8000000080000000ull;  // negated
    }
  }
  const float inv_d = 1.0f / (float)D;
  __nv_bfloat16* out =
      is_q ? a.q_out + t * a.q_heads * D : a.k_out == nullptr ? nullptr : a.k_out + t * a.kv_heads * D;
  __nv_bfloat16* cached = cache_row >= 0 ? a.k_cache + cache_row * a.kv_heads * D : nullptr;

#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * kHeads;
    const uint64_t xa[2] = {unpack2(x[s].a.x), unpack2(x[s].a.y)};
    const uint64_t xb[2] = {unpack2(x[s].b.x), unpack2(x[s].b.y)};
    uint64_t sq = mul2(xa[0], xa[0]);
    sq = fma2(xa[1], xa[1], sq);
    sq = fma2(xb[0], xb[0], sq);
    sq = fma2(xb[1], xb[1], sq);
    float s0, s1;
    unpair(sq, s0, s1);
    float ss = s0 + s1;
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
    const float r = pos_ok ? rsqrtf(ss * inv_d + a.eps) : 0.f;
    const uint64_t r2 = pair(r, r);
    uint64_t ya[2], yb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ya[i] = mul2(xa[i], wc_a[i]);
      yb[i] = mul2(xb[i], wc_b[i]);
      if (kAll || rot) {  // an infinity must not reach a channel it is not rotated with
        ya[i] = fma2(xb[i], ws_b[i], ya[i]);
        yb[i] = fma2(xa[i], ws_a[i], yb[i]);
      }
      ya[i] = mul2(ya[i], r2);
      yb[i] = mul2(yb[i], r2);
    }
    Pairs o;
    o.a = make_uint2(pack2(ya[0]), pack2(ya[1]));
    o.b = make_uint2(pack2(yb[0]), pack2(yb[1]));
    if (!pos_ok) o.a = o.b = make_uint2(0, 0);
    if (!active || h >= heads) continue;
    if (out != nullptr) store_pairs<kInterleaved>(out + h * D, ca, cb, o);
    if (cached != nullptr) store_pairs<kInterleaved>(cached + h * D, ca, cb, o);
  }
  report(a.err, err);
}

template <int kLanes, bool kInterleaved, bool kAll>
int launch(NormRopeArgs a, cudaStream_t stream) {
  constexpr int kSteps = 4;
  constexpr int kUnit = kSteps * (32 / kLanes);
  a.q_units = (a.q_heads + kUnit - 1) / kUnit;
  a.kv_units = (a.kv_heads + kUnit - 1) / kUnit;
  a.units = a.q_units + a.kv_units * (a.v_cache != nullptr ? 2 : 1);
  const int64_t warps = (int64_t)a.num_tokens * a.units;
  const int64_t ctas = (warps * 32 + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  return launch_pdl(norm_rope_kernel<kLanes, kInterleaved, kAll, kSteps>, (unsigned)ctas, kThreads,
                    0, stream, a);
}

template <int kLanes>
int launch(const NormRopeArgs& a, bool interleaved, cudaStream_t stream) {
  const bool all = a.rotary_dim == a.head_dim;
  if (interleaved) return all ? launch<kLanes, true, true>(a, stream) : launch<kLanes, true, false>(a, stream);
  return all ? launch<kLanes, false, true>(a, stream) : launch<kLanes, false, false>(a, stream);
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
  const auto over_either = [&](const void* p, int64_t bytes) {
    return overlap(q_out, qo, p, bytes) || overlap(k_out, ko, p, bytes);
  };
  if (over_either(q_weight, (int64_t)head_dim * 2) || over_either(k_weight, (int64_t)head_dim * 2) ||
      over_either(positions, (int64_t)num_tokens * 8) ||
      over_either(cos_sin, max_position * rotary_dim * 4) ||
      (cached && over_either(slot_mapping, (int64_t)num_tokens * 8)))
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
                 cached ? (int64_t)layer * num_blocks : 0, num_blocks, block_size,
                 BlockDiv::make(block_size), slot_mapping, d_err, 0, 0, 0};
  if (head_dim <= 64) return launch<8>(a, interleaved != 0, stream);
  if (head_dim <= 128) return launch<16>(a, interleaved != 0, stream);
  return launch<32>(a, interleaved != 0, stream);
}
