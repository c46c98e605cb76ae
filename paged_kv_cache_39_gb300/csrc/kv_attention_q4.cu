// kv_attention_q4.cu -- attention of one query token per request over the 4-bit
// paged cache.
//
// Mathematics.  Request r attends the positions [start, end) that its block table
// maps to a block of the pool.  With codes u, group scales a (of K) and b (of V)
//   s_p = scale sum_j a_pj (sum_{c in j} q_c (u_pc - 8)),   w_p = 2^(s_p - ref)
//   o_c = sum_p (w_p b_pj) (u_pc - 8) / sum_p w_p           (c in group j)
// so the group scales never touch the codes: K's multiply the 32-bit partial sum of
// their group, V's the weight.  u - 8 is exact in fp16, q is made exact by a power of
// two per head (2^-24 of its largest channel is lost at most), w b is rounded to fp16
// (2^-11 of it: fewer bits than that would double the output's own rounding error).  So that it
// stays inside fp16 whatever the scales are, a query has a running reference, an integer at or
// above its largest logit when last raised, and for each of its channel groups a power of two f_j:
// the product's operand is w b f_j, the largest one of a group is 2^7 at least, and reference and f
// are set anew when a weight or an operand passes 2^15.  An operand below 2^-14 keeps fewer bits,
// at most 2^-32 of its own group's largest (or 2^-137 outright) is lost then: groups and tokens of very different scales
// do not cost each other bits.  f_j is taken off when a segment ends; sums are held in 32 bits.
//
// GPU shape.  The bytes of the cache bound this: a group's query rows, 4, 8 or 16 at a time, read
// each of them, far under a matrix unit tile of 128 rows, so the products go through the warp's
// own m16n8k16 instruction with tokens (of K) or channels (of V) as its 16 rows and the
// group's query heads as its 8 columns.  The positions of all requests are cut into units of
// 32, and the warps into gangs of one warp per KV head (at most 16): gang i takes the units
// [i C, (i+1) C) whatever requests they belong to, so every warp reads the same number of
// bytes however long the contexts are, and the heads of a block, which lie side by side in
// memory, are read at about the same time (the loads alone: 220 us for 1.2 GB; 237 with a warp
// per equal share of all (head, position) instead).  A warp's units come through a ring of
// kStages in shared memory, filled with cp.async by table lookups made a window of 8 units
// ahead, and nothing but the warp itself waits for them.  A warp whose range ends inside a
// (request, head) leaves its sums in the workspace; a second kernel joins those.
//
// Measured (32 query heads, 8 KV heads of 128 channels): 8 contexts of 131072 tokens 229 us
// (1.21 GB, 5.3 TB/s), 256 contexts of 512 to 4096 tokens 136 us (0.64 GB, 4.7 TB/s), one of 1009
// 9.1 us, of which the second kernel is 2.5, one of 16384 13.9.  A unit of 32 tokens of one head is
// 4608 bytes and about 650 instructions of a warp, half of them on the logic pipe (taking the codes
// apart); with 12 warps an SM issues 2.35 of 4 a cycle.  The groups' powers of two are 2 % of it.  16 warps of 128 registers spill (253 us), 14 leave two
// of the four schedulers one warp short (312 us).
//
// Layout of a unit in shared memory.  Row rho of the K product's 16 is token pi(rho) =
// (rho >> 1) + 4 (rho & 1): its transpose then gives lane t the tokens t, t + 4, t + 8,
// t + 12 it holds of V.  K rows are stored in the order of rho and V's 16-byte pieces
// are xor-ed with the token, which makes every shared-memory read free of bank conflicts.
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "kv_q4.cuh"

namespace kvp {
namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 1;                  // per SM: 12 warps of 168 registers, 3 per scheduler
constexpr int kStages = 3;
constexpr int kUnit = 32;                 // tokens of a unit
constexpr int kWindow = 8 * kUnit;        // tokens of a table lookup
constexpr int kJoinRows = 4;              // rows of a CTA of the join, where a warp takes one
constexpr float kRefStart = -1e30f;       // below every logit, and finite
constexpr float kLimit = 32768.0f;        // a weight or an operand above this sets references anew
constexpr int kTarget = 7;                // log2 of what a group's largest operand is set to, at least
constexpr int kFactorMax = 127 + 112;     // exponent field of the largest f: f times a weight is finite

struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  Q4Layout at;
  int32_t num_blocks32;  // num_blocks, or the largest block id + 1 there can be
  BlockDiv div;
  const int32_t* table;
  int32_t stride;
  const int32_t* start;
  const int32_t* end;
  int32_t num_reqs, q_heads, group;
  int32_t passes;   // groups of NQ query heads per KV head
  int32_t gang;     // warps that take the same positions of neighbouring (KV head, pass)
  int32_t gangs;
  float scale_log2;
  __nv_bfloat16* out;
  int64_t* offsets;  // [num_reqs + 1] units before each request (written by CTA 0)
  float* parts;      // [workers][2][NQ][D + 2]: sums, reference, weight sum
  int32_t* err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// A power of two by its exponent field.
__device__ __forceinline__ float pow2(int field) { return __uint_as_float((uint32_t)field << 23); }
// The powers of two of a lane's two columns, as bf16.
__device__ __forceinline__ uint32_t pack_pow2(int field0, int field1) {
  return (uint32_t)field0 << 7 | (uint32_t)field1 << 23;
}
__device__ __forceinline__ int field_of(uint32_t f, int k) { return (f >> (k ? 23 : 7)) & 0xff; }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1, float c0, float c1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// Four pairs of codes (nibble n of the low and of the high half of x) as fp16 operands.  A
// masked nibble is an fp16 of its own, below the normal range: u 2^-24, or u 2^-20 one nibble
// up (odd n).
constexpr float kCode = 16777216.f;  // 2^24
__device__ __forceinline__ void codes_raw(uint32_t x, uint32_t (&f)[4]) {
  const uint32_t y = x >> 8;
  f[0] = x & 0x000f000fu;
  f[1] = x & 0x00f000f0u;
  f[2] = y & 0x000f000fu;
  f[3] = y & 0x00f000f0u;
}
// K's go into the product as they are (one logic instruction a pair): odd channels meet a
// query divided by 16, and the 8 that belongs off every code is what the accumulator starts
// from, -8 sum q.  V's become (u - 8) 2^-9 with one exact fma a pair: their sums run over
// thousands of tokens, where an 8 taken off at the end would cost the bits of the result.
constexpr float kCentred = 512.f;
__device__ __forceinline__ void codes_centred(uint32_t x, uint32_t (&f)[4]) {
  const __half2 m0 = __float2half2_rn(32768.f), m1 = __float2half2_rn(2048.f);
  const __half2 sub = __float2half2_rn(-8.f / kCentred);
  codes_raw(x, f);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const __half2 a = __hfma2(*reinterpret_cast<const __half2*>(&f[n]), n & 1 ? m1 : m0, sub);
    f[n] = *reinterpret_cast<const uint32_t*>(&a);
  }
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The G bf16 scales of a token.
template <int G>
__device__ __forceinline__ void load_scales(const unsigned char* p, float (&f)[G]) {
  uint32_t w[G / 2];
  if constexpr (G == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int j = 0; j < G; j += 2) {
    f[j] = __uint_as_float(w[j / 2] << 16);
    f[j + 1] = __uint_as_float(w[j / 2] & 0xffff0000u);
  }
}

template <int G>
struct Stage {
  static constexpr int kCodes = kUnit * 16 * G;  // bytes of K (or V) codes
  static constexpr int kScales = kUnit * 2 * G;
  static constexpr int kBytes = 2 * kCodes + 2 * kScales;
};

// A request's span, cut at the end of its table row (so the work is bounded by the table
// whatever the span says), in units of 32 positions that start at multiples of 32.  Blocks
// are multiples of 8 tokens, so 8 aligned positions always lie in one block.
struct Span {
  int32_t lo, hi;    // positions [lo, hi)
  int32_t first;     // unit of position lo
  int32_t units;     // 0: nothing to attend
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int r, uint32_t& err) {
  const int64_t row = (int64_t)a.stride * a.at.block_size;
  const int32_t s0 = a.start[r], s1 = a.end[r];
  if (s0 < 0 || s1 < s0 || (s1 > row && s1 > s0)) err |= KV_ERR_BAD_POSITION;
  Span s;
  s.lo = s0;
  s.hi = (int32_t)min((int64_t)s1, row);
  const bool any = s0 >= 0 && s.hi > s0;
  s.first = any ? s0 / kUnit : 0;
  s.units = any ? (s.hi - 1) / kUnit - s.first + 1 : 0;
  return s;
}
// The unit a worker loads next: positions [p, p + 32) of request r for seg = head * passes +
// pass; `left` units of this (request, seg) are still to load, this one included.
struct Cursor {
  int r, seg, left;
  int32_t p;
  Span span;
  // Steps to the next unit; true when that is the first of another segment.
  __device__ __forceinline__ bool next(const AttnArgs& a, int segs) {
    p += kUnit;
    if (--left > 0) return false;
    seg += a.gang;
    if (seg >= segs) {
      seg %= a.gang;
      uint32_t ignore = 0;
      do {
        if (++r >= a.num_reqs) {  // behind the last unit: not loaded
          left = 1;
          p = 0;
          span.lo = span.hi = 0;
          return true;
        }
        span = span_of(a, r, ignore);
      } while (span.units == 0);
    }
    left = span.units;
    p = span.first * kUnit;
    return true;
  }
};

// kPack (at most 4 query heads per KV head): the 8 columns of the products are the 4 heads for
// tokens 0-15 of the unit and the 4 heads for tokens 16-31, so the work between the products is
// done once per unit.  Query fragments hold zeros in the other half's columns; each half has
// sums and references of its own, added when the segment ends.
template <int G, int NT, bool kPack>
__global__ void __launch_bounds__(kThreads, kCtas) attention_q4_kernel(AttnArgs a) {
  constexpr int D = 32 * G, NQ = kPack ? 4 : 8 * NT;
  constexpr int kHalves = kPack ? 2 : 1;  // token halves that share the columns
  using S = Stage<G>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_before[kThreads];  // units before each thread's share of the requests
  __shared__ int64_t s_warp[kWarps];
  __shared__ int64_t s_total;
  // per unit in the ring: positions that count; request; seg; 1: first of its segment, 2: last
  __shared__ int4 s_unit[kWarps][kStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.at.kv_heads, segs = H * a.passes;
  const int rounds = segs / a.gang;  // times a gang goes over a request's positions
  pdl_allow_next();
  pdl_wait();

  // ---- every CTA: where the requests' units begin
  const int per = (a.num_reqs + kThreads - 1) / kThreads;
  uint32_t err = 0;
  {
    const int r_lo = min(a.num_reqs, tid * per), r_hi = min(a.num_reqs, r_lo + per);
    uint32_t span_err = 0;
    int64_t mine = 0;
    for (int r = r_lo; r < r_hi; ++r) mine += (int64_t)span_of(a, r, span_err).units * rounds;
    if (blockIdx.x == 0) err |= span_err;
    const int64_t incl = warp_inclusive_scan<int64_t>(mine);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    s_before[tid] = before;
    if (tid == kThreads - 1) s_total = before + mine;
    if (blockIdx.x == 0) {
      uint32_t ignore = 0;
      int64_t at = before;
      for (int r = r_lo; r < r_hi; ++r) {
        a.offsets[r] = at;
        at += (int64_t)span_of(a, r, ignore).units * rounds;
      }
      if (tid == kThreads - 1) a.offsets[a.num_reqs] = at;
    }
    __syncthreads();
  }
  // neighbouring workers on neighbouring SMs: little work spreads over all of them
  const int worker = warp * gridDim.x + blockIdx.x;
  // requests without a position: zeros
  for (int r = worker; r < a.num_reqs; r += gridDim.x * kWarps) {
    uint32_t ignore = 0;
    if (span_of(a, r, ignore).units > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)r * a.q_heads * D);
    for (int i = lane; i < a.q_heads * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
  }
  const int64_t total = s_total;
  const int64_t share = (total + a.gangs - 1) / a.gangs;
  const int my_gang = worker / a.gang;
  const int64_t first = my_gang * share;
  if (my_gang >= a.gangs || first >= total) {
    report(a.err, err);
    return;
  }
  int64_t count = min(share, total - first);

  // ---- this worker's first unit
  Cursor load;
  {
    int lo = 0, hi = kThreads;  // last thread whose share begins at or before `first`
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_before[mid] <= first) lo = mid; else hi = mid;
    }
    int r = lo * per;
    int64_t at = s_before[lo];
    uint32_t ignore = 0;
    load.span = span_of(a, r, ignore);
    while (at + (int64_t)load.span.units * rounds <= first) {
      at += (int64_t)load.span.units * rounds;
      load.span = span_of(a, ++r, ignore);
    }
    const int64_t rest = first - at;
    const int round = (int)(rest / load.span.units);
    const int unit = (int)(rest - (int64_t)round * load.span.units);
    load.r = r;
    load.seg = round * a.gang + (worker - my_gang * a.gang);
    load.left = load.span.units - unit;
    load.p = (load.span.first + unit) * kUnit;
  }

  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * kStages * S::kBytes;
  const unsigned char* ring_p = smem + warp * kStages * S::kBytes;
  // this lane's piece of every 512 bytes of codes: token tok, 16-byte chunk c, and where K and V
  // pieces go (see the layout above)
  const int piece_tok = lane / G, piece_c = lane % G;
  const uint32_t k_dst = ring + 16 * piece_c +
                         (2 * (piece_tok & 3) + ((piece_tok >> 2) & 1) + (piece_tok & 8)) * (16 * G);
  const uint32_t v_dst = ring + S::kCodes + piece_tok * (16 * G) +
                         16 * (G == 4 ? piece_c ^ (2 * ((piece_tok >> 1) & 1)) : piece_c);
  const uint32_t s_dst = ring + 2 * S::kCodes + lane * 16;
  const int T = a.at.block_size;
  const int step_off = kUnit % T;
  const uint32_t rec16 = (uint32_t)(T / 8) * (9 * G);  // T (16 G + 2 G) / 16
  const uint32_t block16 = rec16 * (uint32_t)H;

  // ---- loads.  Blocks are looked up for 8 units at once, lane l for positions 8 l .. 8 l + 7
  // of the window, and one window ahead: a unit's copies never wait for its table entry.
  // Offsets are in 16-byte pieces of the layer (32 bits: checked on the host); the codes of 8
  // tokens are 8 G pieces, their scales G.
  const uint8_t* const k_lane = a.k_cache + 16 * (G == 4 ? lane : lane & 15);
  const int64_t k_to_v = a.v_cache - a.k_cache;
  const uint8_t* const s_lane = (lane < 4 * G ? a.k_cache : a.v_cache) + 16 * (lane % G);
  const int s_run = lane % (4 * G) / G;
  int32_t window, blocks, blocks_next;
  int32_t off;       // first token of run lane & 3 in its block
  uint32_t head_at;  // the head's record in a block
  auto look_up = [&](int64_t from) {
    const int64_t run = from + 8 * lane;
    if (run >= load.span.hi || run + 7 < load.span.lo) return kNull;
    int64_t lb, ignore;
    a.div.divmod(run, lb, ignore);
    return a.table[(int64_t)load.r * a.stride + lb];
  };
  auto open_segment = [&]() {
    window = load.p;
    blocks = look_up(window);
    blocks_next = look_up((int64_t)window + kWindow);
    int64_t lb, first_off;
    a.div.divmod((int64_t)load.p + 8 * (lane & 3), lb, first_off);
    off = (int32_t)first_off;
    head_at = (uint32_t)(load.seg / a.passes) * rec16;
  };
  auto issue = [&](int stage) {
    if (load.p - window >= kWindow) {
      window += kWindow;
      blocks = blocks_next;
      blocks_next = look_up((int64_t)window + kWindow);
    }
    // lane l stands for run l & 3 of the unit
    const int32_t nb = __shfl_sync(kFull, blocks, (load.p - window) / 8 + (lane & 3));
    const uint32_t runs =
        __ballot_sync(kFull, (uint32_t)nb - 1u < (uint32_t)a.num_blocks32 - 1u) & 15u;
    const uint32_t rec = (uint32_t)nb * block16 + head_at;
    const uint32_t codes = rec + (uint32_t)off * G;
    const uint32_t scales = rec + (uint32_t)T * G + (uint32_t)(off >> 3) * G;
    const uint32_t at = stage * S::kBytes;
    uint32_t mask = kFull;
    if (runs == 15u && load.p >= load.span.lo && load.p + kUnit - 1 < load.span.hi) {
#pragma unroll
      for (int i = 0; i < G; ++i) {  // 32 / G tokens each: lane's piece is 16 lane bytes into them
        const uint32_t c = __shfl_sync(kFull, codes, G == 4 ? i : 2 * i + (lane >> 4));
        const uint8_t* src = k_lane + (uint64_t)c * 16;
        copy16(k_dst + at + i * 512, src);
        copy16(v_dst + at + i * 512, src + k_to_v);
      }
      // scales: K's by the first 4 G lanes, V's by the next, 16 bytes each like the codes
      const uint32_t c = __shfl_sync(kFull, scales, s_run);
      if (G == 4 || lane < 8 * G) copy16(s_dst + at, s_lane + (uint64_t)c * 16);
    } else {  // a span's edge, or a run without a block: nothing is read for that run
      if (!((runs >> (lane & 3)) & 1u) && nb != kNull) err |= KV_ERR_BAD_BLOCK;
      // 4 validity bits of the runs, each spread over its 8 positions
      mask = ((runs * 0x00204081u) & 0x01010101u) * 0xffu;
      const int32_t skip = load.span.lo - load.p, stop = load.span.hi - load.p;
      if (skip > 0) mask &= kFull << skip;
      if (stop < kUnit) mask &= stop > 0 ? (1u << stop) - 1u : 0u;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int run = G == 4 ? i : 2 * i + (lane >> 4);
        const uint32_t c = __shfl_sync(kFull, codes, run);
        const uint8_t* src = k_lane + (uint64_t)c * 16;
        if ((runs >> run) & 1u) {
          copy16(k_dst + at + i * 512, src);
          copy16(v_dst + at + i * 512, src + k_to_v);
        }
      }
      const uint32_t c = __shfl_sync(kFull, scales, s_run);
      if ((G == 4 || lane < 8 * G) && ((runs >> s_run) & 1u))
        copy16(s_dst + at, s_lane + (uint64_t)c * 16);
    }
    if (lane == 0)
      s_unit[warp][stage] = make_int4((int)mask, load.r, load.seg,
                                      (load.p == load.span.first * kUnit ? 1 : 0) |
                                          (load.left == 1 ? 2 : 0));
    off += step_off;
    if (off >= T) off -= T;
    if (load.next(a, segs)) open_segment();
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  open_segment();
  int64_t to_load = count;
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) {
    if (to_load > 0) {
      issue(s);
      --to_load;
    }
    commit();
  }

  uint32_t qf[kHalves][NT][G][2][2];  // query fragments
  float qc[NT][2];           // what a logit of this lane's two columns is multiplied with
  float qs[NT][G][2];        // -8 2^-24 sum q of a group, for those columns
  float o[NT][2 * G][4];     // sums: rows = channels, columns = query heads
  float ref[NT][2], sum[NT][2];
  uint32_t fj[NT][G];        // f of each group, for those columns
  bool fresh = true, from_start = false;
  const int tok = (g >> 1) + 4 * (g & 1);               // this lane's token of each 8
  const uint32_t half_mask = g < 4 ? kFull : 0u;        // kPack: columns of tokens 0-15
  const int half_tok = kPack ? 16 * (t >> 1) + tok : tok;

  int stage = 0;
#pragma unroll 1
  for (; count > 0; --count) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    if (to_load > 0) {
      issue(stage == 0 ? kStages - 1 : stage - 1);  // where the unit before this one was
      --to_load;
    }
    commit();

    const int4 now = s_unit[warp][stage];
    const uint32_t mask = (uint32_t)now.x;
    if (fresh) {  // a new (request, head, pass)
      fresh = false;
      from_start = now.w & 1;
      const int head = now.z / a.passes, pass = now.z - head * a.passes;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int qi = pass * NQ + 8 * n + (kPack ? g & 3 : g);
        float x[G][8], top = 0.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (qi < a.group)
            v = *reinterpret_cast<const uint4*>(a.q + now.y * a.q_stride +
                                                (int64_t)(head * a.group + qi) * D + 32 * j + 8 * t);
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[j][2 * k] = __uint_as_float(e[k] << 16);
            x[j][2 * k + 1] = __uint_as_float(e[k] & 0xffff0000u);
            top = fmaxf(top, fmaxf(fabsf(x[j][2 * k]), fabsf(x[j][2 * k + 1])));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^(13-e) with e the exponent of the largest channel (1 for rows of zeros, and for 2^100 up)
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const bool usual = e > -100 && e < 100;
        const float down = usual ? __uint_as_float((uint32_t)(140 - e) << 23) : 1.f;
        const float up = usual ? __uint_as_float((uint32_t)(114 + e) << 23) : 1.f;
#pragma unroll
        for (int j = 0; j < G; ++j) {
          float total = 0.f;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float by = k ? down * 0.0625f : down;
              const uint32_t f = pack_f16(x[j][2 * s + k] * by, x[j][4 + 2 * s + k] * by);
              if (kPack) {
                qf[0][n][j][s][k] = f & half_mask;
                qf[kHalves - 1][n][j][s][k] = f & ~half_mask;
              } else {
                qf[0][n][j][s][k] = f;
              }
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
              total += (k ? 16.f : 1.f) * (v.x + v.y);
            }
          total += __shfl_xor_sync(kFull, total, 1);
          total += __shfl_xor_sync(kFull, total, 2);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            qs[n][j][k] = __shfl_sync(kFull, total, 4 * (2 * t + k)) * (-8.f / kCode);
        }
        // column 2 t + k is the query head of lanes 4 (2 t + k) ..
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // in the order that neither overflows nor loses bits early, and inside the normal range: a
          // factor of zero or infinity would make NaN of hidden (infinite) or zero products
          const float u = __shfl_sync(kFull, up, 4 * (2 * t + k)), c = a.scale_log2;
          qc[n][k] = fminf(fmaxf(c > 1.f ? u * c * kCode : u * (c * kCode), FLT_MIN), FLT_MAX);
          ref[n][k] = kRefStart;
          sum[n][k] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < G; ++j) fj[n][j] = pack_pow2(kFactorMax, kFactorMax);
#pragma unroll
        for (int m = 0; m < 2 * G; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[n][m][k] = 0.f;
      }
    }

    const unsigned char* base = ring_p + stage * S::kBytes;
    // K codes of 16 tokens (half u) times the query fragments, group by group
    auto logits = [&](int u, int h, float (&acc)[G][NT][4], bool start) {
      uint32_t x[2][G];  // per row: the group's codes of g' = 2 t (low half) and 2 t + 1 (high)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const unsigned char* row = base + (16 * u + 8 * r + g) * (16 * G);
        if constexpr (G == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * t);
          x[r][0] = __byte_perm(w.x, w.z, 0x5410);
          x[r][1] = __byte_perm(w.x, w.z, 0x7632);
          x[r][2] = __byte_perm(w.y, w.w, 0x5410);
          x[r][3] = __byte_perm(w.y, w.w, 0x7632);
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * t);
          x[r][0] = __byte_perm(w.x, w.y, 0x5410);
          x[r][1] = __byte_perm(w.x, w.y, 0x7632);
        }
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        uint32_t lo[4], hi[4];
        codes_raw(x[0][j], lo);
        codes_raw(x[1][j], hi);
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (start)
            mma16816_from(acc[j][n], a0, qf[h][n][j][0][0], qf[h][n][j][0][1], qs[n][j][0],
                          qs[n][j][1]);
          else
            mma16816(acc[j][n], a0, qf[h][n][j][0][0], qf[h][n][j][0][1]);
          mma16816(acc[j][n], a1, qf[h][n][j][1][0], qf[h][n][j][1][1]);
        }
      }
    };
    // From the products to the weights times V's scales, as fragments of the second product;
    // `first_tok`: this lane's first token of the unit (the second is 8 further).
    auto weights = [&](int first_tok, const float (&acc)[G][NT][4], uint32_t (&b)[G][NT][2]) {
      float ks[2][G], vs[2][G], s[NT][4], w[NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned char* sc = base + 2 * S::kCodes + (first_tok + 8 * h) * (2 * G);
        load_scales<G>(sc, ks[h]);
        load_scales<G>(sc + S::kScales, vs[h]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[n][k] = acc[0][n][k] * ks[k >> 1][0];
#pragma unroll
          for (int j = 1; j < G; ++j) s[n][k] = fmaf(acc[j][n][k], ks[k >> 1][j], s[n][k]);
        }
      // hidden positions: no weight, and whatever bits the ring holds as scales (codes are finite
      // whatever they are)
      if (mask != kFull) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!((mask >> (first_tok + 8 * h)) & 1u)) {
#pragma unroll
            for (int j = 0; j < G; ++j) vs[h][j] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][2 * h] = s[n][2 * h + 1] = -INFINITY;
          }
      }
      float most = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[n][k] = ex2(fmaf(s[n][k], qc[n][k & 1], -ref[n][k & 1]));
          most = fmaxf(most, w[n][k]);
        }
      // w b f as fp16; the largest magnitude of all in `top`
      __half2 top = __float2half2_rn(0.f);
      auto operands = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const float f0 = __uint_as_float(fj[n][j] << 16), f1 = __uint_as_float(fj[n][j] & 0xffff0000u);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              b[j][n][h] = pack_f16(w[n][2 * h] * f0 * vs[h][j], w[n][2 * h + 1] * f1 * vs[h][j]);
              top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&b[j][n][h])));
            }
          }
      };
      operands();
      if (__any_sync(kFull, most > kLimit || !__hble2(top, __float2half2_rn(kLimit)))) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          int drop[2];  // log2 of what a reference rises by
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float z = fmaxf(s[n][k] * qc[n][k], s[n][k + 2] * qc[n][k]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) z = fmaxf(z, __shfl_xor_sync(kFull, z, d));
            const float up = fmaxf(ref[n][k], ceilf(z)), by = up - ref[n][k];
            drop[k] = by < 400.f ? (int)by : 400;
            sum[n][k] *= ex2(-by);
            ref[n][k] = up;
            w[n][k] = ex2(fmaf(s[n][k], qc[n][k], -up));
            w[n][k + 2] = ex2(fmaf(s[n][k + 2], qc[n][k], -up));
          }
#pragma unroll
          for (int j = 0; j < G; ++j) {
            // the largest w b of these tokens, its upper 16 bits, of both columns
            uint32_t m[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              m[k] = __float_as_uint(fmaxf(w[n][k] * fabsf(vs[0][j]), w[n][k + 2] * fabsf(vs[1][j])));
            uint32_t both = __byte_perm(m[0], m[1], 0x7632);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) both = __vmaxu2(both, __shfl_xor_sync(kFull, both, d));
            int field[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int was = field_of(fj[n][j], k);
              // what leaves the sums as they are, unless the largest needs it lower
              field[k] = min(min(was + drop[k], kFactorMax), 2 * 127 + kTarget - field_of(both, k));
              const int by = field[k] - was - drop[k];  // <= 0
              const float f = by > -127 ? pow2(127 + by) : 0.f;
#pragma unroll
              for (int m = 2 * j; m < 2 * j + 2; ++m) {
                o[n][m][k] *= f;
                o[n][m][k + 2] *= f;
              }
            }
            fj[n][j] = pack_pow2(field[0], field[1]);
          }
        }
        operands();
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sum[n][0] += w[n][0] + w[n][2];
        sum[n][1] += w[n][1] + w[n][3];
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) b[j][n][h] = transpose8x8(b[j][n][h]);
      }
    };
    // V codes of 16 tokens (half u) times weight fragments; columns outside `keep` count as 0
    auto values = [&](int u, const uint32_t (&b)[G][NT][2], uint32_t keep) {
      uint32_t vw[4][G / 2];  // tokens t, t + 4, t + 8, t + 12
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned char* row = base + S::kCodes + (16 * u + t + 4 * q) * (16 * G);
        if constexpr (G == 4) {
          const uint2 v =
              *reinterpret_cast<const uint2*>(row + ((g >> 1) ^ (t & 2)) * 16 + (g & 1) * 8);
          vw[q][0] = v.x;
          vw[q][1] = v.y;
        } else {
          vw[q][0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
        }
      }
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        uint32_t lo[4], hi[4];
        codes_centred(__byte_perm(vw[0][j / 2], vw[1][j / 2], sel), lo);
        codes_centred(__byte_perm(vw[2][j / 2], vw[3][j / 2], sel), hi);
        const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]}, a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t b0 = kPack ? times(b[j][n][0], keep) : b[j][n][0];
          const uint32_t b1 = kPack ? times(b[j][n][1], keep) : b[j][n][1];
          mma16816(o[n][2 * j], a0, b0, b1);
          mma16816(o[n][2 * j + 1], a1, b0, b1);
        }
      }
    };

    float acc[G][NT][4];
    uint32_t b[G][NT][2];
    if constexpr (kPack) {
      logits(0, 0, acc, true);
      logits(1, 1, acc, false);
      weights(half_tok, acc, b);
      values(0, b, half_mask & 0x3c003c00u);
      values(1, b, ~half_mask & 0x3c003c00u);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        logits(u, 0, acc, true);
        weights(16 * u + tok, acc, b);
        values(u, b, kFull);
      }
    }

    // ---- the segment or this worker's share of it is done
    const bool last = now.w & 2;
    if (last || count == 1) {
      fresh = true;
      const int head = now.z / a.passes, pass = now.z - head * a.passes;
      const bool whole = last && from_start;
      float* part = a.parts + ((int64_t)worker * 2 + (from_start ? 1 : 0)) * NQ * (D + 2);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const float f = pow2(2 * 127 - field_of(fj[n][j], k));
#pragma unroll
            for (int m = 2 * j; m < 2 * j + 2; ++m) {
              o[n][m][k] *= f;
              o[n][m][k + 2] *= f;
            }
          }
          float l = sum[n][k];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(kFull, l, d);
          if (kPack) {  // columns 4.. are the same heads, over the other half of the tokens
            const float other = __shfl_xor_sync(kFull, ref[n][k], 2);
            const float top = fmaxf(ref[n][k], other), f = ex2(ref[n][k] - top);
            l *= f;
            l += __shfl_xor_sync(kFull, l, 2);
            ref[n][k] = top;
#pragma unroll
            for (int m = 0; m < 2 * G; ++m)
#pragma unroll
              for (int i = k; i < 4; i += 2) {
                o[n][m][i] *= f;
                o[n][m][i] += __shfl_xor_sync(kFull, o[n][m][i], 2);
              }
          }
          const int qi = 8 * n + 2 * t + k;  // in this pass
          if (qi >= NQ || pass * NQ + qi >= a.group) continue;
          if (whole) {
            const float inv = l == 0.f ? 0.f : kCentred / l;
            __nv_bfloat16* out =
                a.out + ((int64_t)now.y * a.q_heads + head * a.group + pass * NQ + qi) * D;
#pragma unroll
            for (int j = 0; j < G; ++j) {
              const __nv_bfloat162 p0 =
                  __floats2bfloat162_rn(o[n][2 * j][k] * inv, o[n][2 * j][k + 2] * inv);
              const __nv_bfloat162 p1 =
                  __floats2bfloat162_rn(o[n][2 * j + 1][k] * inv, o[n][2 * j + 1][k + 2] * inv);
              *reinterpret_cast<uint2*>(out + 32 * j + 4 * g) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
            }
          } else {
            float* p = part + qi * (D + 2);
#pragma unroll
            for (int j = 0; j < G; ++j) {
              float2* d = reinterpret_cast<float2*>(p + 32 * j + 4 * g);
              d[0] = make_float2(o[n][2 * j][k], o[n][2 * j][k + 2]);
              d[1] = make_float2(o[n][2 * j + 1][k], o[n][2 * j + 1][k + 2]);
            }
            if (g == 0) *reinterpret_cast<float2*>(p + D) = make_float2(ref[n][k], l);
          }
        }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  report(a.err, err);
}

// Join: out = sum_i 2^(ref_i - top) o_i / sum_i 2^(ref_i - top) l_i over the parts the
// workers left of one (request, query head); which worker holds which part follows from the
// offsets alone.  W warps take the parts in turn, the first kFirst of them and then 8 at a
// time, so that a long row of parts costs few round trips: the 228 of one context of 16384
// tokens take 4 us with 16 warps, 11 with 8 warps and 4 parts at a time.  Each lane has D / 32
// channels.
template <int G, int NQ, int W>
__global__ void __launch_bounds__(W == 1 ? 32 * kJoinRows : 32 * W) join_q4_kernel(AttnArgs a) {
  constexpr int D = 32 * G, kFirst = W == 1 ? 2 : 4, kMore = 8;
  __shared__ float s_o[W][D], s_l[W], s_top[W];
  pdl_allow_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
  const unsigned row = W == 1 ? blockIdx.x * kJoinRows + (threadIdx.x >> 5) : blockIdx.x;
  if (W == 1 && row >= (unsigned)a.num_reqs * (unsigned)a.q_heads) return;
  const int r = row / (unsigned)a.q_heads, qh = row - r * a.q_heads;
  const int rounds = a.at.kv_heads * a.passes / a.gang;
  const int64_t at = a.offsets[r], after = a.offsets[r + 1], total = a.offsets[a.num_reqs];
  if (after == at) return;  // zeros, already written
  const int head = qh / a.group, qi = qh - head * a.group;
  const int seg = head * a.passes + qi / NQ, round = seg / a.gang;
  int64_t i0, i1;
  if (total <= INT32_MAX) {  // 32-bit divisions are a third of a microsecond faster
    const uint32_t units = (uint32_t)(after - at) / (uint32_t)rounds;
    const uint32_t share = ((uint32_t)total + a.gangs - 1) / (uint32_t)a.gangs;
    const uint32_t lo = (uint32_t)at + round * units;
    i0 = lo / share, i1 = (lo + units - 1) / share;
  } else {
    const int64_t units = (after - at) / rounds, share = (total + a.gangs - 1) / a.gangs;
    const int64_t lo = at + round * units;
    i0 = lo / share, i1 = (lo + units - 1) / share;
  }
  if (i0 == i1) return;    // one worker saw it whole
  const float* parts = a.parts + (int64_t)(qi % NQ) * (D + 2);
  constexpr int64_t kPart = NQ * (D + 2);

  float acc[G] = {}, l = 0.f, top = kRefStart;
  auto add = [&](auto batch, int64_t i) {  // the parts i, i + W, ..
    constexpr int kBatch = decltype(batch)::value;
    float ref[kBatch], sum[kBatch], v[kBatch][G];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t x = i + b * W;
      const float* p = parts + (2 * (x * a.gang + (seg - round * a.gang)) + (x == i0 ? 1 : 0)) * kPart;
      const bool in = x <= i1;
      ref[b] = in ? p[D] : kRefStart;
      sum[b] = in ? p[D + 1] : 0.f;
#pragma unroll
      for (int j = 0; j < G; ++j) v[b][j] = in ? p[32 * j + lane] : 0.f;
    }
    float up = top;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) up = fmaxf(up, ref[b]);
    const float f = ex2(top - up);
    top = up;
    l *= f;
#pragma unroll
    for (int j = 0; j < G; ++j) acc[j] *= f;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float g = ex2(ref[b] - up);
      l = fmaf(sum[b], g, l);
#pragma unroll
      for (int j = 0; j < G; ++j) acc[j] = fmaf(v[b][j], g, acc[j]);
    }
  };
  int64_t next = i0 + warp;
  add(std::integral_constant<int, kFirst>{}, next);
#pragma unroll 1
  for (next += kFirst * W; next <= i1; next += kMore * W) add(std::integral_constant<int, kMore>{}, next);
  __nv_bfloat16* out = a.out + ((int64_t)r * a.q_heads + qh) * D;
  if constexpr (W == 1) {
    const float inv = l == 0.f ? 0.f : kCentred / l;
#pragma unroll
    for (int j = 0; j < G; ++j) out[32 * j + lane] = __float2bfloat16_rn(acc[j] * inv);
  } else {
    if (lane == 0) s_top[warp] = top, s_l[warp] = l;
#pragma unroll
    for (int j = 0; j < G; ++j) s_o[warp][32 * j + lane] = acc[j];
    __syncthreads();
    if (threadIdx.x >= D) return;
    const int some = (int)min((int64_t)W, i1 - i0 + 1);  // warps that had a part
    for (int w = 0; w < some; ++w) top = fmaxf(top, s_top[w]);
    float sum = 0.f, o = 0.f;
#pragma unroll 4
    for (int w = 0; w < some; ++w) {
      const float f = ex2(s_top[w] - top);
      sum = fmaf(f, s_l[w], sum);
      o = fmaf(f, s_o[w][threadIdx.x], o);
    }
    out[threadIdx.x] = __float2bfloat16_rn(o * (sum == 0.f ? 0.f : kCentred / sum));
  }
}

// Query heads a warp takes at once: 4, 8, or 16 (the cache is read once for all of them).  16 heads
// of 128 channels do not fit in its registers: two passes of 8 instead, whose second reads come from
// the L2 (64 contexts of 4096 tokens, 4 KV heads: 72 us against 88 with 16 and spills; of 64
// channels, 38 with 16).
int columns(int group, int head_dim) {
  return group > 8 && head_dim == 64 ? 16 : group > 4 ? 8 : 4;
}
int worker_count() { return sm_count() * kCtas * kWarps; }
// The largest divisor of the (KV head, pass) pairs up to 16.
int gang_size(int segs) {
  int g = segs < 16 ? segs : 16;
  while (segs % g != 0) --g;
  return g;
}
int64_t offsets_bytes(int32_t num_reqs) { return ((int64_t)(num_reqs + 1) * 8 + 127) / 128 * 128; }

template <int G, int NQ>
int launch(const AttnArgs& a, cudaStream_t stream) {
  auto kernel = attention_q4_kernel<G, NQ == 16 ? 2 : 1, NQ == 4>;
  constexpr int smem = kWarps * kStages * Stage<G>::kBytes;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return KV_ECUDA;
  const int rc = launch_pdl(kernel, worker_count() / kWarps, kThreads, smem, stream, a);
  if (rc != KV_OK) return rc;
  // about so many parts a row: more warps where they are many
  const unsigned rows = (unsigned)a.num_reqs * (unsigned)a.q_heads;
  const int parts = a.gangs / a.num_reqs;
  if (parts >= 32) return launch_pdl(join_q4_kernel<G, NQ, 16>, rows, 32 * 16, 0, stream, a);
  if (parts >= 8) return launch_pdl(join_q4_kernel<G, NQ, 8>, rows, 32 * 8, 0, stream, a);
  return launch_pdl(join_q4_kernel<G, NQ, 1>, (rows + kJoinRows - 1) / kJoinRows, 32 * kJoinRows,
                    0, stream, a);
}

template <int G>
int launch(const AttnArgs& a, cudaStream_t stream) {
  switch (columns(a.group, 32 * G)) {
    case 4: return launch<G, 4>(a, stream);
    case 8: return launch<G, 8>(a, stream);
    default: return G == 2 ? launch<2, 16>(a, stream) : KV_EUNSUPPORTED;
  }
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int64_t kv_attention_q4_workspace(int32_t num_reqs, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim) {
  if (num_reqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_q_heads % num_kv_heads != 0)
    return KV_EINVAL;
  if (num_reqs > KV_MAX_GATHER_REQS || num_q_heads > 4096 || (head_dim != 64 && head_dim != 128))
    return KV_EUNSUPPORTED;
  const int group = num_q_heads / num_kv_heads;
  return offsets_bytes(num_reqs) +
         (int64_t)worker_count() * 2 * columns(group, head_dim) * (head_dim + 2) * 4;
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
  const Q4Layout at{0, num_blocks, block_size, num_kv_heads, head_dim};
  // the kernel addresses a layer in 16-byte pieces of 32 bits
  const int64_t block_bytes = at.record_bytes() * num_kv_heads;
  if (num_blocks > ((int64_t)1 << 36) / block_bytes) return KV_EUNSUPPORTED;
  const int64_t row = (int64_t)num_q_heads * head_dim;
  const int64_t need = kv_attention_q4_workspace(num_reqs, num_q_heads, num_kv_heads, head_dim);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
    return KV_EINVAL;
  const int64_t spans = (int64_t)num_reqs * 4, cache = block_bytes * num_blocks;
  const auto over_input = [&](const void* p, int64_t bytes) {
    return overlap(p, bytes, query, ((num_reqs - 1) * query_stride + row) * 2) ||
           overlap(p, bytes, block_table, spans * table_stride) || overlap(p, bytes, span_start, spans) ||
           overlap(p, bytes, span_end, spans) ||
           overlap(p, bytes, static_cast<const char*>(k_cache) + layer * cache, cache) ||
           overlap(p, bytes, static_cast<const char*>(v_cache) + layer * cache, cache);
  };
  if (over_input(out, num_reqs * row * 2) || over_input(workspace, need) ||
      overlap(out, num_reqs * row * 2, workspace, need))
    return KV_EINVAL;
  const int group = num_q_heads / num_kv_heads;
  const int passes = (group + columns(group, head_dim) - 1) / columns(group, head_dim);
  const int gang = gang_size(num_kv_heads * passes);
  const int64_t layer_at = layer * cache;
  AttnArgs a{static_cast<const __nv_bfloat16*>(query), query_stride,
             static_cast<const uint8_t*>(k_cache) + layer_at,
             static_cast<const uint8_t*>(v_cache) + layer_at, at,
             (int32_t)(num_blocks < INT32_MAX ? num_blocks : INT32_MAX),
             BlockDiv::make(block_size), block_table, table_stride, span_start, span_end, num_reqs,
             num_q_heads, group, passes, gang, worker_count() / gang,
             fminf(scale * 1.44269504088896340736f, FLT_MAX),
             static_cast<__nv_bfloat16*>(out), static_cast<int64_t*>(workspace),
             reinterpret_cast<float*>(static_cast<char*>(workspace) + offsets_bytes(num_reqs)),
             d_err};
  return head_dim == 128 ? launch<4>(a, stream) : launch<2>(a, stream);
}
