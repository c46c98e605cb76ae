// kv_cache_q4.cu -- write of new K/V rows into the 4-bit paged cache, and the
// gather of spans of it as bf16 rows.
//
// Mathematics (layout in kv_q4.cuh).  For a group of 32 channels x of one row
//   s = bf16(max|x| / 7),  code = round(x / s) + 8  (nearest, ties to even),
// read back as (code - 8) * s.  round(x / s) is found without a division: x and s have 8
// significant bits each, so x / s, at most 7 (1 + 2^-8), is either a tie k + 1/2 or more than
// 2^-10 away from every one, and the integer q nearest to x times an approximate 1 / s (within
// 2^-22) is right unless x / s is a tie.  Then, and only then, 2 |x - q s| == s, which is exact in
// 32 bits; groups with a tie are done again value by value.  No clamp is needed.
// 8 lanes quantise a head's K and V rows, each lane finding one of the 8 groups' scales: 8192
// tokens of 8 x 128 take 11.6 us (43 MB), bound by the instructions (14.3 with every scale found
// by 8 lanes, 25 with divisions and value by value); 256 tokens 2.7 us in a graph.
#include "kv_q4.cuh"

namespace kvp {
namespace {

constexpr float kRound = 12582920.0f;  // 1.5 * 2^23 + 8: adding it rounds to an integer and
                                       // leaves the code, the integer + 8, in the low bits

struct WriteArgs {
  const __nv_bfloat16* key;
  const __nv_bfloat16* value;
  int64_t key_stride, value_stride;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  int32_t num_tokens;
  Q4Layout at;
  BlockDiv div;
  int32_t* err;
};

constexpr int kWriteThreads = 128;

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max / 7 as the fp32 quotient: a product with the rounded reciprocal, then its remainder, exact in
// an fma, once more times the reciprocal (Markstein's correction, IBM J. Res. Dev. 34, 1990).  The
// remainder of a tiny value would leave the normal range: divided.
__device__ __forceinline__ float over_seven(float x) {
  if (x < 1e-18f) return __fdiv_rn(x, 7.0f);
  const float c = 1.0f / 7.0f, q = x * c;
  return fmaf(fmaf(-7.0f, q, x), c, q);
}
// The codes of 4 values of scale s, ties to even: the slow way, for groups that hold a tie.
__device__ __noinline__ uint32_t codes_with_ties(float v0, float v1, float v2, float v3, float s,
                                                 float inv) {
  const float v[4] = {v0, v1, v2, v3};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = fmaf(v[i], inv, kRound);
    int code = __float_as_int(t) & 15;
    const float r = fmaf(kRound - t, s, v[i]);  // x - q s
    if (fabsf(r) * 2.f == s && (code & 1)) code += r > 0.f ? 1 : -1;
    c |= (uint32_t)code << (4 * i);
  }
  return c;
}

// The scale of the group whose largest magnitude has the bits m.
struct Scale {
  uint32_t bits;  // bf16
  float half;     // half of it, or -1 where every code is 8 (zeros, or NaN and infinity)
  float inv;      // about 1 / scale, or 0 there
};
__device__ __forceinline__ Scale scale_of(uint32_t m) {
  const __nv_bfloat16 b = __float2bfloat16_rn(over_seven(__uint_as_float(m)));
  const float s = __bfloat162float(b);
  Scale r{__bfloat16_as_ushort(b), 0.5f * s, 0.f};
  if (s < 1.17549435e-38f) r.half = -1.f, r.bits = 0u;   // below the normal range: a group of zeros
  if (m >= 0x7f800000u) r.half = -1.f, r.bits = 0x7fc0u;  // infinity or NaN: the group reads as NaN
  if (r.half > 0.f) r.inv = rcp_approx(s);
  return r;
}

// One row of one head by 8 lanes: lane g holds channels 32 j + 4 g .. + 3; lane `from` + j of the
// warp holds the scale of group j.
template <int G>
__device__ __forceinline__ void quantise_row(const uint2 (&x)[G], const Scale& mine, int from,
                                             uint8_t* codes, int g, bool store) {
  uint32_t half[G];   // 4 codes of each group
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float tie = __shfl_sync(kFull, mine.half, from + j), s = tie + tie;
    const float inv = __shfl_sync(kFull, mine.inv, from + j);
    const uint64_t v[2] = {pair(__uint_as_float(x[j].x << 16), __uint_as_float(x[j].x & 0xffff0000u)),
                           pair(__uint_as_float(x[j].y << 16), __uint_as_float(x[j].y & 0xffff0000u))};
    const uint64_t inv2 = pair(inv, inv), s2 = pair(s, s), round2 = pair(kRound, kRound);
    const uint64_t minus = pair(-1.f, -1.f);
    uint32_t c = 0;
    bool tied = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t t = fma2(v[i], inv2, round2);
      const uint64_t r = fma2(fma2(t, minus, round2), s2, v[i]);  // x - q s
      float t0, t1, r0, r1;
      unpair(t, t0, t1);
      unpair(r, r0, r1);
      tied |= fabsf(r0) == tie || fabsf(r1) == tie;
      // the low 16 bits: the float's own bits above the code are multiples of 2^22
      c += (__float_as_uint(t0) + 16u * __float_as_uint(t1)) << (8 * i);
    }
    if (tied) {
      float v0, v1, v2, v3;
      unpair(v[0], v0, v1);
      unpair(v[1], v2, v3);
      c = codes_with_ties(v0, v1, v2, v3, s, inv);
    }
    half[j] = c;
  }
  if (!store) return;
  if constexpr (G == 4)
    *reinterpret_cast<uint2*>(codes + 8 * g) = make_uint2(__byte_perm(half[0], half[1], 0x5410),
                                                          __byte_perm(half[2], half[3], 0x5410));
  else
    *reinterpret_cast<uint32_t*>(codes + 4 * g) = __byte_perm(half[0], half[1], 0x5410);
}

// Largest magnitudes of the row's groups as integers (NaN > infinity > every finite value), two
// groups to a word, over the 8 lanes.
template <int G>
__device__ __forceinline__ void largest(const uint2 (&x)[G], uint32_t (&top)[G / 2]) {
#pragma unroll
  for (int j = 0; j < G; j += 2) {
    const uint32_t a = __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu);
    const uint32_t b = __vmaxu2(x[j + 1].x & 0x7fff7fffu, x[j + 1].y & 0x7fff7fffu);
    uint32_t m = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFull, m, k));
    top[j / 2] = m;
  }
}

template <int G>
__global__ void __launch_bounds__(kWriteThreads) write_q4_kernel(WriteArgs a) {
  pdl_allow_next();
  pdl_wait();
  const int g = threadIdx.x & 7;
  const int64_t item = ((int64_t)blockIdx.x * kWriteThreads + threadIdx.x) >> 3;
  const int H = a.at.kv_heads;
  const bool in = item < (int64_t)a.num_tokens * H;
  const int64_t t = !in ? 0 : item <= INT32_MAX ? (uint32_t)item / (uint32_t)H : item / H;
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
    int64_t b, rest;
    a.div.divmod(s, b, rest);
    if (b == kNull) {
      err |= KV_ERR_NULL_WRITE;
    } else if (b >= a.at.num_blocks) {
      err |= KV_ERR_BAD_SLOT;
    } else {
      const int32_t off = (int32_t)rest;
      const int64_t rec = a.at.record(b, h);
      kc = a.k_cache + rec + a.at.codes(off);
      vc = a.v_cache + rec + a.at.codes(off);
      ks = a.k_cache + rec + a.at.scales(off);
      vs = a.v_cache + rec + a.at.scales(off);
      store = true;
    }
  }
  uint32_t k_top[G / 2], v_top[G / 2];
  largest<G>(k, k_top);
  largest<G>(v, v_top);
  // each lane finds one scale: K's groups in lanes 0 .. G - 1 of the 8, V's in the next G
  const bool is_v = g & G;
  const int group = g % G;
  uint32_t word = is_v ? v_top[0] : k_top[0];
  if constexpr (G == 4) {
    if (group & 2) word = is_v ? v_top[1] : k_top[1];
  }
  const Scale mine = scale_of(group & 1 ? word & 0xffff0000u : word << 16);
  if (store && g < 2 * G)
    reinterpret_cast<uint16_t*>(is_v ? vs : ks)[group] = (uint16_t)mine.bits;
  const int from = threadIdx.x & 24;
  quantise_row<G>(k, mine, from, kc, g, store);
  quantise_row<G>(v, mine, from + G, vc, g, store);
  report(a.err, err);
}

// ---------------------------------------------------------------------------
// Gather.  As the bf16 gather: every CTA scans the span lengths into packed output offsets,
// then warps walk the output rows, kGatherRows at a time.  Eight lanes stand for two of the
// rows and go through their heads, so the block and the position in it are resolved once per
// row and a head is one addition to each address.  The output's bytes bound it (256 of 328 a
// head at 128 channels): 94833 rows of 8 x 128, K and V, take 82 us, 6.1 TB/s of these bytes, 0.91 of
// what a plain copy reaches.  The conversion is
// 5 instructions for two values, in bf16 pairs (11 one by one, and 86 us).

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 8;
constexpr size_t kGatherStaticSmem = sizeof(int64_t) * (kGatherThreads / 32);

struct GatherArgs {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  Q4Layout at;
  BlockDiv div;
  const int32_t* table;
  int32_t stride;
  const int32_t* g0;
  const int32_t* g1;
  int32_t num_reqs;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int64_t out_rows;
  int32_t part_log2, part_heads;  // 2^part_log2 warps share a group of rows, part_heads each
  int32_t* err;
};

// The four codes of h (16 bits) times scale s (bf16, in both halves), as two bf16 pairs.  A
// nibble under the exponent of 128 is 128 + u; less 136 it is u - 8, both exact, and the product
// is the only rounding.
__device__ __forceinline__ uint2 values4(uint32_t h, uint32_t s, uint32_t exponent) {
  const uint32_t t = h | h << 12;  // nibbles 1 and 3 again, where the upper half has 0 and 2
  uint32_t a, b;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(a) : "r"(t), "r"(exponent));
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(b) : "r"(t >> 8), "r"(exponent));
  const __nv_bfloat162 off = __floats2bfloat162_rn(-136.f, -136.f);
  const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&s);
  const __nv_bfloat162 x = __hmul2_rn(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), off), scale);
  const __nv_bfloat162 y = __hmul2_rn(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&b), off), scale);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// One row of one head by 8 lanes: lane l holds the codes of g = 2 (l & 3) and the next g, of
// which it stores the groups j = l >> 2 and j + 2: 8 channels, 16 bytes, each, so that the 8
// lanes write whole 128-byte lines.
template <int G>
struct PackedRow {
  uint32_t c[G], s[G / 2];
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales) {
    if constexpr (G == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(codes);
      const uint2 w = *reinterpret_cast<const uint2*>(scales);
      c[0] = u.x, c[1] = u.y, c[2] = u.z, c[3] = u.w, s[0] = w.x, s[1] = w.y;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(codes);
      c[0] = u.x, c[1] = u.y;
      s[0] = *reinterpret_cast<const uint32_t*>(scales);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < G; ++i) c[i] = 0x88888888u;
#pragma unroll
    for (int i = 0; i < G / 2; ++i) s[i] = 0u;
  }
  // high: this lane's groups are in the words' upper halves
  __device__ __forceinline__ void store(__nv_bfloat16* row, bool high, uint32_t exponent) const {
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
      const uint32_t f = __byte_perm(s[i], 0, high ? 0x3232 : 0x1010);
      const uint2 x = values4(__byte_perm(c[i], 0, high ? 0x4432 : 0x4410), f, exponent);
      const uint2 y = values4(__byte_perm(c[G / 2 + i], 0, high ? 0x4432 : 0x4410), f, exponent);
      st_stream(reinterpret_cast<uint4*>(row + 64 * i), make_uint4(x.x, x.y, y.x, y.y));
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

  const int H = a.at.kv_heads;
  const bool high = lane & 4;
  const int channel = (high ? 32 : 0) + 8 * (lane & 3);  // this lane's first
  const int64_t rec = a.at.record_bytes();
  uint32_t exponent;  // 128 in both halves; opaque, so that it stays one operand of a lop3
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(exponent));
  const int64_t warp0 = ((int64_t)blockIdx.x * kGatherThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kGatherThreads) >> 5;
  const int64_t items = ((rows + kGatherRows - 1) / kGatherRows) << a.part_log2;
  for (int64_t item = warp0; item < items; item += nwarps) {
    const int64_t o0 = (item >> a.part_log2) * kGatherRows;
    const int h0 = (int)(item & ((1 << a.part_log2) - 1)) * a.part_heads;
    const int h1 = min(H, h0 + a.part_heads);
    const int nr = (int)(rows - o0 < kGatherRows ? rows - o0 : kGatherRows);
    // rows lane / 8 and lane / 8 + 4: where their codes and scales are for head h0, or zero rows
    const uint8_t *kc[2], *vc[2];
    int64_t to_scales[2];
    bool in[2], full[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int64_t o = o0 + (lane >> 3) + 4 * n;
      in[n] = (lane >> 3) + 4 * n < nr;
      full[n] = false;
      kc[n] = vc[n] = nullptr;
      to_scales[n] = 0;
      if (!in[n]) continue;
      const int r = find_span64(s_off, R, o);
      const int64_t p = (int64_t)s_start[r] + (o - s_off[r]);
      int64_t lb, off;
      a.div.divmod(p, lb, off);
      if (lb >= a.stride) {
        err |= KV_ERR_BAD_POSITION;
        continue;
      }
      const int64_t b = a.table[(int64_t)r * a.stride + lb];
      if (b == kNull) continue;
      if (b < 0 || b >= a.at.num_blocks) {
        err |= KV_ERR_BAD_BLOCK;
        continue;
      }
      full[n] = true;
      const int64_t at = a.at.record(b, h0) + a.at.codes((int32_t)off) + 4 * G * (lane & 3);
      kc[n] = a.k_cache + at;
      vc[n] = a.v_cache + at;
      to_scales[n] = a.at.scales((int32_t)off) - a.at.codes((int32_t)off) - 4 * G * (lane & 3);
    }
    __nv_bfloat16* ko = a.k_out + ((o0 + (lane >> 3)) * H + h0) * (32 * G) + channel;
    __nv_bfloat16* vo = a.v_out + ((o0 + (lane >> 3)) * H + h0) * (32 * G) + channel;
    const int64_t four = (int64_t)4 * H * (32 * G);
#pragma unroll 2
    for (int h = h0; h < h1; ++h) {
      PackedRow<G> k[2], v[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        k[n].zero();
        v[n].zero();
        if (full[n]) {
          k[n].load(kc[n], kc[n] + to_scales[n]);
          v[n].load(vc[n], vc[n] + to_scales[n]);
          kc[n] += rec;
          vc[n] += rec;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (in[n]) {
          k[n].store(ko + n * four, high, exponent);
          v[n].store(vo + n * four, high, exponent);
        }
      }
      ko += 32 * G;
      vo += 32 * G;
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
              BlockDiv::make(block_size), d_err};
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
               BlockDiv::make(block_size), block_table, table_stride, gather_start, gather_end, num_reqs,
               static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), out_rows,
               0, 0, d_err};
  auto kernel = head_dim == 128 ? gather_q4_kernel<4> : gather_q4_kernel<2>;
  const size_t smem = sizeof(int64_t) * (num_reqs + 1) + sizeof(int32_t) * num_reqs;
  const int64_t rows_per_cta = (kGatherThreads / 32) * kGatherRows;
  const int64_t need = (out_rows + rows_per_cta - 1) / rows_per_cta;
  const int64_t cap = (int64_t)sm_count() * (2048 / kGatherThreads);
  // Few rows: their heads are spread over more warps, until the GPU is full or a warp has one
  // (256 rows of 8 heads: 8.3 -> 3.9 us).
  while ((2 << a.part_log2) <= num_kv_heads && (need << a.part_log2) * 2 <= cap) ++a.part_log2;
  a.part_heads = (num_kv_heads + (1 << a.part_log2) - 1) >> a.part_log2;
  const int64_t parts = need << a.part_log2;
  const int grid = (int)(need < 1 ? 1 : (parts < cap ? parts : cap));
  if (smem + kGatherStaticSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return KV_ECUDA;
  return launch_pdl(kernel, grid, kGatherThreads, smem, stream, a);
}
