// kv_cache_q4.cu -- write of new K/V rows into the 4-bit paged cache, and the
// gather of spans of it as bf16 rows.
//
// Mathematics (layout in kv_q4.cuh).  For a group of 32 channels x of one row
//   s = bf16(max|x| / 7),  code = round(x / s) + 8  (nearest, ties to even),
// read back as (code - 8) * s.  round(x / s) is found without a division: with
// t = x * (1/s) rounded to an integer q, x / s is within 2^-23 of t, and as x
// and s have 8 significant bits each, x / s is either a tie (k + 1/2) or more
// than 2^-13 away from one.  So q is right unless 2 |x - q s| == s, which is
// tested exactly (q s and the difference fit 32 bits), and a tie goes to even.
// |x / s| <= 7 (1 + 2^-8), so no clamp is needed.
#include "kv_q4.cuh"

namespace kvp {
namespace {

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

struct WriteArgs {
  const __nv_bfloat16* key;
  const __nv_bfloat16* value;
  int64_t key_stride, value_stride;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  int32_t num_tokens;
  Q4Layout at;
  int32_t* err;
};

constexpr int kWriteThreads = 128;

// One row of one head by 8 lanes: lane g holds channels 32 j + 4 g .. + 3.
template <int G>
__device__ __forceinline__ void quantise_row(const uint2 (&x)[G], uint8_t* codes, uint8_t* scales,
                                             int g, bool store) {
  uint32_t half[G];   // 4 codes of each group
  uint32_t sbits[G];  // bf16 scales
#pragma unroll
  for (int j = 0; j < G; ++j) {
    // magnitudes as integers: NaN > infinity > every finite value
    const uint32_t m2 = __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu);
    uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) m = max(m, __shfl_xor_sync(kFull, m, k));
    const float amax = __uint_as_float(m << 16);
    const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
    float s = __bfloat162float(sb);
    sbits[j] = __bfloat16_as_ushort(sb);
    float inv = 0.f;
    if (m >= 0x7f80u) {          // an infinity or a NaN: the whole group reads as NaN
      sbits[j] = 0x7fc0u;
    } else if (s < 1.17549435e-38f) {  // scale below the normal range: a group of zeros
      sbits[j] = 0u;
    } else {
      inv = __frcp_rn(s);
    }
    const float v[4] = {__uint_as_float(x[j].x << 16), __uint_as_float(x[j].x & 0xffff0000u),
                        __uint_as_float(x[j].y << 16), __uint_as_float(x[j].y & 0xffff0000u)};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int ti = 0;
      if (inv != 0.f) {
        const float t = fmaf(v[i], inv, kRound);
        ti = __float_as_int(t);
        const float r = fmaf(kRound - t, s, v[i]);  // x - q s, exact
        if (fabsf(r) * 2.f == s && (ti & 1)) ti += r > 0.f ? 1 : -1;
      }
      c |= (uint32_t)((ti + 8) & 15) << (4 * i);
    }
    half[j] = c;
  }
  if (!store) return;
  if constexpr (G == 4) {
    *reinterpret_cast<uint2*>(codes + 8 * g) =
        make_uint2(half[0] | half[1] << 16, half[2] | half[3] << 16);
    if (g == 0)
      *reinterpret_cast<uint2*>(scales) =
          make_uint2(sbits[0] | sbits[1] << 16, sbits[2] | sbits[3] << 16);
  } else {
    *reinterpret_cast<uint32_t*>(codes + 4 * g) = half[0] | half[1] << 16;
    if (g == 0) *reinterpret_cast<uint32_t*>(scales) = sbits[0] | sbits[1] << 16;
  }
}

template <int G>
__global__ void __launch_bounds__(kWriteThreads) write_q4_kernel(WriteArgs a) {
  pdl_allow_next();
  pdl_wait();
  const int g = threadIdx.x & 7;
  const int64_t item = ((int64_t)blockIdx.x * kWriteThreads + threadIdx.x) >> 3;
  const int H = a.at.kv_heads, T = a.at.block_size;
  const bool in = item < (int64_t)a.num_tokens * H;
  const int64_t t = in ? item / H : 0;
  const int h = (int)(item - t * H);
  uint2 k[G], v[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    k[j] = v[j] = make_uint2(0, 0);
    if (in) {
      k[j] = *reinterpret_cast<const uint2*>(a.key + t * a.key_stride + h * (32 * G) + 32 * j + 4 * g);
      v[j] =
          *reinterpret_cast<const uint2*>(a.value + t * a.value_stride + h * (32 * G) + 32 * j + 4 * g);
    }
  }
  uint32_t err = 0;
  uint8_t *kc = nullptr, *vc = nullptr, *ks = nullptr, *vs = nullptr;
  const int64_t s = in ? a.slots[t] : -1;
  bool store = false;
  if (s >= 0) {
    const int64_t b = s / T;
    if (b == kNull) {
      err |= KV_ERR_NULL_WRITE;
    } else if (b >= a.at.num_blocks) {
      err |= KV_ERR_BAD_SLOT;
    } else {
      const int32_t off = (int32_t)(s - b * T);
      const int64_t rec = a.at.record(b, h);
      kc = a.k_cache + rec + a.at.codes(off);
      vc = a.v_cache + rec + a.at.codes(off);
      ks = a.k_cache + rec + a.at.scales(off);
      vs = a.v_cache + rec + a.at.scales(off);
      store = true;
    }
  }
  quantise_row<G>(k, kc, ks, g, store);
  quantise_row<G>(v, vc, vs, g, store);
  report(a.err, err);
}

// ---------------------------------------------------------------------------
// Gather.  As the bf16 gather: every CTA scans the span lengths into packed
// output offsets, then warps walk the output rows, kGatherRows at a time: lane
// i resolves the slot of row i, and 8 lanes turn one (row, head) of K and of V
// into bf16.

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 8;
constexpr size_t kGatherStaticSmem = sizeof(int64_t) * (kGatherThreads / 32);

struct GatherArgs {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  Q4Layout at;
  const int32_t* table;
  int32_t stride;
  const int32_t* g0;
  const int32_t* g1;
  int32_t num_reqs;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t out_rows;
  int32_t* err;
};

// Two codes (nibbles 4 i and 4 i + 4 of c) as bf16 values times scale s.
__device__ __forceinline__ uint32_t value2(uint32_t c, int i, float s) {
  const float lo = (float)((int)((c >> (4 * i)) & 15u) - 8) * s;
  const float hi = (float)((int)((c >> (4 * i + 4)) & 15u) - 8) * s;
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int G>
struct PackedRow {
  uint32_t c[G / 2], s[G / 2];
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int g) {
    if constexpr (G == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(codes + 8 * g);
      const uint2 w = *reinterpret_cast<const uint2*>(scales);
      c[0] = u.x, c[1] = u.y, s[0] = w.x, s[1] = w.y;
    } else {
      c[0] = *reinterpret_cast<const uint32_t*>(codes + 4 * g);
      s[0] = *reinterpret_cast<const uint32_t*>(scales);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) c[i] = 0x88888888u, s[i] = 0u;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, int g) const {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const uint32_t h = j & 1 ? c[j / 2] >> 16 : c[j / 2] & 0xffffu;
      const float f = __uint_as_float(j & 1 ? s[j / 2] & 0xffff0000u : s[j / 2] << 16);
      *reinterpret_cast<uint2*>(row + 32 * j + 4 * g) = make_uint2(value2(h, 0, f), value2(h, 2, f));
    }
  }
};

template <int G>
__global__ void __launch_bounds__(kGatherThreads) gather_q4_kernel(GatherArgs a) {
  pdl_allow_next();
  pdl_wait();
  extern __shared__ int64_t smem[];
  int64_t* s_off = smem;                                                 // [num_reqs + 1]
  int32_t* s_start = reinterpret_cast<int32_t*>(smem + a.num_reqs + 1);  // [num_reqs]
  __shared__ int64_t s_warp_sum[kGatherStaticSmem / sizeof(int64_t)];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, R = a.num_reqs;
  uint32_t err = 0;

  // packed output offsets: exclusive scan of the span lengths
  const int per = (R + kGatherThreads - 1) / kGatherThreads;
  const int r_lo = min(R, (int)threadIdx.x * per), r_hi = min(R, r_lo + per);
  int64_t local = 0;
  uint32_t span_err = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const int32_t s0 = a.g0[r], s1 = a.g1[r];
    const bool ok = s0 >= 0 && s1 >= s0;
    if (!ok) span_err |= KV_ERR_BAD_POSITION;
    s_start[r] = s0;
    local += ok ? (int64_t)(s1 - s0) : 0;
  }
  const int64_t incl = warp_inclusive_scan<int64_t>(local);
  if (lane == 31) s_warp_sum[wid] = incl;
  __syncthreads();
  int64_t run = incl - local;
  for (int w = 0; w < wid; ++w) run += s_warp_sum[w];
  for (int r = r_lo; r < r_hi; ++r) {
    s_off[r] = run;
    const int32_t s0 = s_start[r], s1 = a.g1[r];
    run += (s0 >= 0 && s1 >= s0) ? (int64_t)(s1 - s0) : 0;
  }
  if (threadIdx.x == kGatherThreads - 1) s_off[R] = run;
  __syncthreads();
  const int64_t total = s_off[R];
  if (blockIdx.x == 0) {
    err |= span_err;
    if (threadIdx.x == 0 && total > a.out_rows) err |= KV_ERR_OUT_OF_SPACE;
  }
  const int64_t rows = total < a.out_rows ? total : a.out_rows;

  const int H = a.at.kv_heads, T = a.at.block_size, g = lane & 7;
  const int64_t warp0 = ((int64_t)blockIdx.x * kGatherThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kGatherThreads) >> 5;
  for (int64_t o0 = warp0 * kGatherRows; o0 < rows; o0 += nwarps * kGatherRows) {
    const int nr = (int)(rows - o0 < kGatherRows ? rows - o0 : kGatherRows);
    int64_t slot = -1;  // lane i < nr: the slot of row o0 + i, or -1 for a zero row
    if (lane < nr) {
      const int64_t o = o0 + lane;
      const int r = find_span64(s_off, R, o);
      const int64_t p = (int64_t)s_start[r] + (o - s_off[r]);
      const int64_t lb = p / T;
      if (lb >= a.stride) {
        err |= KV_ERR_BAD_POSITION;
      } else {
        const int64_t b = a.table[(int64_t)r * a.stride + lb];
        if (b != kNull) {
          if (b < 0 || b >= a.at.num_blocks) err |= KV_ERR_BAD_BLOCK;
          else slot = b * T + (p - lb * T);
        }
      }
    }
    const int items = nr * H;
    for (int i0 = 0; i0 < items; i0 += 8) {  // two (row, head) of K and V per 8 lanes
      PackedRow<G> k[2], v[2];
      int row[2], head[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int i = i0 + 4 * n + (lane >> 3);
        row[n] = i / H;
        head[n] = i - row[n] * H;
        const int64_t s = __shfl_sync(kFull, slot, row[n] & 31);
        k[n].zero();
        v[n].zero();
        if (i < items && s >= 0) {
          const int64_t b = s / T;
          const int32_t off = (int32_t)(s - b * T);
          const int64_t rec = a.at.record(b, head[n]);
          k[n].load(a.k_cache + rec + a.at.codes(off), a.k_cache + rec + a.at.scales(off), g);
          v[n].load(a.v_cache + rec + a.at.codes(off), a.v_cache + rec + a.at.scales(off), g);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int i = i0 + 4 * n + (lane >> 3);
        if (i >= items) continue;
        const int64_t at = ((o0 + row[n]) * H + head[n]) * (32 * G);
        k[n].store(a.k_out + at, g);
        v[n].store(a.v_out + at, g);
      }
    }
  }
  report(a.err, err);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_cache_write_q4(const void* key, int64_t key_stride, const void* value,
                                 int64_t value_stride, void* k_cache, void* v_cache,
                                 const int64_t* slot_mapping, int32_t num_tokens, int32_t layer,
                                 int32_t num_layers, int64_t num_blocks, int32_t block_size,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t* d_err,
                                 kv_stream_t stream) {
  const int rc = q4_checks(k_cache, v_cache, layer, num_layers, num_blocks, block_size,
                           num_kv_heads, head_dim, d_err);
  if (rc != KV_OK) return rc;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (num_tokens < 0 || key_stride < row || value_stride < row) return KV_EINVAL;
  if (key_stride % 8 != 0 || value_stride % 8 != 0) return KV_EUNSUPPORTED;
  if (num_tokens == 0) return KV_OK;
  if (key == nullptr || value == nullptr || k_cache == nullptr || v_cache == nullptr ||
      slot_mapping == nullptr || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(slot_mapping, 8))
    return KV_EINVAL;
  const int64_t ctas =
      ((int64_t)num_tokens * num_kv_heads * 8 + kWriteThreads - 1) / kWriteThreads;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  WriteArgs a{static_cast<const __nv_bfloat16*>(key), static_cast<const __nv_bfloat16*>(value),
              key_stride, value_stride, static_cast<uint8_t*>(k_cache),
              static_cast<uint8_t*>(v_cache), slot_mapping, num_tokens,
              Q4Layout{(int64_t)layer * num_blocks, num_blocks, block_size, num_kv_heads, head_dim},
              d_err};
  return launch_pdl(head_dim == 128 ? write_q4_kernel<4> : write_q4_kernel<2>, (unsigned)ctas,
                    kWriteThreads, 0, stream, a);
}

extern "C" int kv_cache_gather_q4(const void* k_cache, const void* v_cache, int32_t layer,
                                  int32_t num_layers, int64_t num_blocks, int32_t block_size,
                                  int32_t num_kv_heads, int32_t head_dim,
                                  const int32_t* block_table, int32_t table_stride,
                                  const int32_t* gather_start, const int32_t* gather_end,
                                  int32_t num_reqs, void* k_out, void* v_out, int64_t out_rows,
                                  int32_t* d_err, kv_stream_t stream) {
  const int rc = q4_checks(k_cache, v_cache, layer, num_layers, num_blocks, block_size,
                           num_kv_heads, head_dim, d_err);
  if (rc != KV_OK) return rc;
  if (num_reqs < 0 || out_rows < 0 || table_stride < 0) return KV_EINVAL;
  if (num_reqs > KV_MAX_GATHER_REQS) return KV_EUNSUPPORTED;
  if (num_reqs == 0) return KV_OK;
  if (gather_start == nullptr || gather_end == nullptr || !aligned(gather_start, 4) ||
      !aligned(gather_end, 4) || k_cache == nullptr || v_cache == nullptr)
    return KV_EINVAL;
  if (table_stride > 0 && (block_table == nullptr || !aligned(block_table, 4))) return KV_EINVAL;
  if (out_rows > 0 && (k_out == nullptr || v_out == nullptr || !aligned(k_out, 16) ||
                       !aligned(v_out, 16)))
    return KV_EINVAL;
  GatherArgs a{static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
               Q4Layout{(int64_t)layer * num_blocks, num_blocks, block_size, num_kv_heads, head_dim},
               block_table, table_stride, gather_start, gather_end, num_reqs,
               static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), out_rows,
               d_err};
  auto kernel = head_dim == 128 ? gather_q4_kernel<4> : gather_q4_kernel<2>;
  const size_t smem = sizeof(int64_t) * (num_reqs + 1) + sizeof(int32_t) * num_reqs;
  const int64_t rows_per_cta = (kGatherThreads / 32) * kGatherRows;
  const int64_t need = (out_rows + rows_per_cta - 1) / rows_per_cta;
  const int64_t cap = (int64_t)sm_count() * (2048 / kGatherThreads);
  const int grid = (int)(need < 1 ? 1 : (need < cap ? need : cap));
  if (smem + kGatherStaticSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return KV_ECUDA;
  return launch_pdl(kernel, grid, kGatherThreads, smem, stream, a);
}
