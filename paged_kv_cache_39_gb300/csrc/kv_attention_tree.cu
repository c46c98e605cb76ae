// kv_attention_tree.cu -- attention of a step's rows (drafted trees, or one token) over the
// bf16 paged caches, on the matrix unit.
//
// Mathematics.  Row i of request r sees the positions [start, context) and context + j for the
// bits j of its mask, as far as the block table maps them to a block of the pool:
//   o_i = sum_p w_ip v_p / sum_p w_ip,  w_ip = 2^(c q_i . k_p - ref_i),  c = scale * log2(e),
// in one pass with a running reference, raised (and the sums rescaled) only when a logit passes it by
// more than 8.  Logits, weights, sums and outputs are held in 32 bits; a weight is rounded
// to bf16 for its product with V (the matrix unit takes both operands in one type), at most
// 2^-8 of it; the sum takes it before that.
//
// GPU shape.  All query heads of a group and all rows of a request read the same keys, so
// its rows are packed (row = token * group + head) into tiles of 128, one (kRows = 1) or two at a time.
// With up to 128 rows the cache's bytes bound this: 128 keys of a head of 128 channels are
// 64 KB, 2850 cycles of an SM's share of the memory, and 1024 of the matrix unit however few of
// the tile's rows there are.  Positions are cut into units of 128, and CTAs (one per SM) into gangs
// of one CTA per KV head or so: gang i takes the units [i C, (i+1) C) whatever requests
// they belong to, so every CTA reads the same number of keys however long the contexts are, and
// the heads of a block, which lie side by side in memory, are read at about the same time.  A CTA
// whose range ends inside a (request, head) leaves its sums in the workspace, and a second
// kernel joins those.
//
// Roles by warp (kTma):
//   softmax    one row per thread (two tiles: per two threads, each half of the keys); also the
//              rescale and the output
//   issuer     the matrix instructions: S = Q K^T, then O += P V with P in tensor memory, over the
//              logits it is made of
//   values     checks V of the units that hold the step's rows or a span's end, before the issuer reads it
//   describer  the requests' units in order: which keys are there, each box's place in the pool
//   2 copiers  K and V by TMA boxes of 8 tokens and more into a ring of 128-key tiles in the 128-byte swizzle
//   Q loader
// Blocks that are no multiple of 8 tokens have four copiers in place of the last four, which describe the
// units, look up rows and copy them with cp.async (rows that are no position of the request are
// zeros), and check V themselves.
// Tensor memory: S twice and O twice.  One tile: units take turns with S, so the next scores are
// computed during this softmax, and segments with O.  Two tiles: one S and O each.
//
// Hidden keys.  A hidden logit is replaced, so a NaN there is gone, but 0 * NaN in P V is NaN.
// Hidden from all rows: made zeros.  Hidden from some rows are only the step's
// own rows: their values are checked when they arrive; what is not finite is set to 0 in
// shared memory and its row noted, and the output of a row that sees it looks the value up again.
//
// Measured, with what the rules choose against (32 query and 8 KV heads of 128 channels, block 16):
//   256 contexts of 512 to 4096 tokens, a row each: 357 us, 6.7 TB/s; 8 of 131072, 16 rows each: 633 us,
//   6.8 TB/s (as fast as the card copies); 64 of 512 to 4096, 2 to 25 rows: 123 us, 5.2 TB/s;
//   64 of 4000: 166 us with a row each, 181 with 16, 190 with 32, 233 with 64 (1160 TFLOP/s);
//   16 of 1000 to 8192, 57 to 64 rows, 40 and 5 heads of 64 channels: 85 us (500 TFLOP/s).
//   TMA or cp.async (the same blocks of 16): 357 and 405 us, 633 and 703, 123 and 132, 233 and 333, 85 and 101.
//   Two tiles at a time for more than 128 rows, or one: 233 and 305 us (64 rows), 85 and 110 (the last case).
//   Gangs of up to 8 CTAs, or none: 357 and 376 us, 123 and 135, 64 contexts of 8000 and 64 channels 229 and 285.
//   Two buffers for Q where five tiles (ten of 64 channels) still fit, or one: 195 and 204 us with cp.async
//   (64 x 16 rows), the same with TMA.
//   Q by TMA, or by cp.async from one warp: 254 and 263 us for 64 rows.
// A call has as many passes over the keys as max_rows asks for, 256 rows each, and a request goes through all of
// them: 240 requests with one row and 16 with 64, 512 to 4096 tokens, 32 query heads: 442, 439 and 438 us with 8, 4
// and 2 KV heads (one, two and four passes), 330 + 78, 178 + 76 and 99 + 75 in two calls.
// One tile is bound by memory.  Two are bound by the chain from scores to weights to products and back:
// 4180 cycles a unit, of which the matrix unit works 2048 and the exponential unit 2048; and by the
// instruction cache: the same waits in longer code cost 5 to 10 %.
#include <cuda_bf16.h>

#include <cfloat>

#include "kv_tc.cuh"
#include "kv_tree.cuh"

namespace kvp {
namespace {

constexpr int kTile = 128;             // keys of a unit, rows of a tile
constexpr int kCopiers = 4;            // warps, where they copy; where TMA does:
constexpr int kReaders = 4;            // that read what the describer writes: K's copies, V's, Q, checks
constexpr int kNotes = 8;              // units described ahead (a power of two: 2^3)
constexpr int kBadRing = 16;           // segments whose values are noted
constexpr float kLazy = 8.0f;          // log2 of the most a weight may pass the reference
constexpr float kRefStart = -1e30f;    // of a row with no finite logit yet
constexpr int kSmemMax = 232448;       // of a CTA
constexpr int kJoinThreads = 128;
constexpr int kJoins = 8;              // CTAs of the join to one of the attention
constexpr int kMaxCtas = 2 * kJoinThreads;  // two to a thread of the join

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
  int32_t passes;    // groups of kRows tiles of a request's rows
  int32_t gang;      // CTAs that take the same positions of neighbouring (KV head, pass)
  int32_t gangs;
  int32_t part_rows; // rows of a part in the workspace
  int32_t q_rows;    // rows of a tile's Q in shared memory (a multiple of 8)
  int32_t q_bufs;    // Q of this segment and the next, where there is room
  int32_t q_box;     // kTma: tokens of a tile, where it begins and ends with a token; else 0
  int32_t slots;     // of the ring
  int32_t box;       // tokens of a TMA box (a power of two that divides the block), or 1
  int32_t warps;     // softmax warps of a tile that can have rows
  int4* joins;       // [CTAs]: the segment a CTA began and did not end: request, segment, last gang
  float* parts;      // [CTAs][2][part_rows][DP], then (reference, sum) [CTAs][2][part_rows]
};

// A request's rows and the positions they may see; no unit: nothing to attend.
struct Req {
  int32_t first, count;   // rows
  uint32_t lo, hi, ctx;   // positions [lo, hi); the step's rows begin at ctx
  uint32_t base;          // of the first unit: lo, down to a multiple of a box
  int32_t units;
};
__device__ __forceinline__ Req request(const TreeArgs& a, int r, uint32_t& err) {
  const StepRows rows = step_rows(a.q_start, r, a.num_rows, a.max_rows);
  const int32_t s0 = a.span_start != nullptr ? a.span_start[r] : 0, c = a.context_len[r];
  Req q = {rows.first, rows.count, 0, 0, 0, 0, 0};
  if (rows.count < 0) err |= KV_ERR_BAD_QSL;
  if (rows.count <= 0) return q;
  if (s0 < 0 || c < s0) {
    err |= KV_ERR_BAD_POSITION;
    return q;
  }
  const int64_t reach = (int64_t)a.stride * a.div.size, end = (int64_t)c + rows.count;
  if (end > reach) err |= KV_ERR_BAD_POSITION;
  q.ctx = (uint32_t)c;
  q.lo = (uint32_t)s0;
  q.hi = (uint32_t)(end < reach ? end : reach);
  q.base = q.lo & ~(uint32_t)(a.box - 1);
  q.units = q.hi > q.lo ? (int32_t)((q.hi - q.base + kTile - 1) / kTile) : 0;
  return q;
}

// What the copiers tell the others about a unit, and, with a segment's first unit here, about the
// segment.
struct __align__(16) Note {
  uint32_t valid[4];       // keys that some row may see
  int32_t step;            // the step's row 0 is key `step` of the unit
  int32_t flags;
  int32_t head;
  int32_t seen;            // keys [seen & 255, seen >> 8) of the unit are positions of the request
  int32_t tokens[16];      // kTma: each box's first token in the pool, < 0: none
};
struct __align__(16) SegNote {
  int32_t r, head, pass;
  int32_t first, count;    // the request's rows
  uint32_t ctx;
  int32_t pad[2];
};
// of this CTA's share; of the segment; values to check (kTma); more rows than a tile in this pass
enum Flags { kFirst = 1, kLast = 2, kFromStart = 4, kToEnd = 8, kEdge = 16, kTwo = 32 };

constexpr int kNumBars = 2 * 12 + 2 * kNotes + 2 + 4 + 2 + 2 + 2 + 1 + 2 + 2 * kNotes + 8;
constexpr int kHead = 3 << 10;         // bytes of shared memory before Q
template <int DP>
struct Layout {
  static constexpr int kSlot = kTile * DP * 2;
  static constexpr int kBars = 0;
  static constexpr int kNote = (kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kSegNote = kNote + kNotes * (int)sizeof(Note);
  static constexpr int kBad = kSegNote + kNotes * (int)sizeof(SegNote);
  static constexpr int kMisc = kBad + kBadRing * 8;                // tensor memory, abort; int64_t: all units
  static constexpr int kWords = kMisc + 32;                        // uint32_t[2][2][4][2]: rows that rise
  static constexpr int kTops = kWords + 128;                       // float[2][128]
  static_assert(kTops + 2 * kTile * 4 <= kHead, "");              // Q, then the ring
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A whole warp's wait, bounded: it gives up 1 s after its eighth try, or where another role has (*abort).
// Short code, as there are many of them and 24 warps share the instruction cache.
// It is voted on, so the lanes of a role never part: what they issue takes its
// operands from uniform registers and wants all of them there.
__device__ __forceinline__ uint32_t timer_low() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t tries = 0, t0 = 0;
  bool ok;
#pragma unroll 1
  while (!(ok = mbar_try_wait(bar, parity))) {
    if (*abort != 0) break;
    if (++tries < 8) continue;
    const uint32_t now = timer_low();
    if (tries == 8) t0 = now;
    if (now - t0 > (uint32_t)kWaitLimitNs) {
      *abort = 1;
      break;
    }
  }
  return __all_sync(kFull, ok) != 0;
}

// Threads: the softmax warps (4 for one tile; 8 for each of two, each warp half of the keys), the issuer's
// four, 4 copiers.
template <int kRows>
constexpr int kThreadsOf = 128 * kRows * kRows + 256;

template <int DP, int kRows, bool kTma>
__global__ void __launch_bounds__(kThreadsOf<kRows>, 1)
attention_tree_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<DP>;
  constexpr int kThreads = kThreadsOf<kRows>;
  constexpr int kHalves = kRows;            // softmax warps that share 32 rows
  constexpr int kIssuer = 4 * kRows * kHalves, kCopy = kIssuer + 4;
  // registers of the warpgroups: 384 threads x 168 at launch = 128 x (240 + 104 + 160), 768 x 80 = 128 x
  // (4 x 88 + 64 + 64)
  constexpr int kSoftmaxRegs = kRows == 1 ? 240 : 88, kIssueRegs = kRows == 1 ? 104 : 64;
  constexpr int kCopyRegs = kRows == 1 ? 160 : 64;
  constexpr int kLag = DP == 128 ? 1 : 3;   // units in flight beside the newest: 128 KB with it
  constexpr int kPieces = DP / 8;           // 16-byte pieces of a row
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* full = bars;
  uint64_t* empty = full + 12;
  uint64_t* note_full = empty + 12;
  uint64_t* note_free = note_full + kNotes;
  uint64_t* s_full = note_free + kNotes;    // one tile: by unit & 1; two: by tile
  uint64_t* p_full = s_full + 2;            // the same, by half of the keys
  uint64_t* o_full = p_full + 4;            // one tile: [0], every unit; two: by tile, at a segment's end
  uint64_t* o_free = o_full + 2;            // one tile: by segment & 1; two: by tile
  uint64_t* q_free = o_free + 2;            // by segment % q_bufs
  uint64_t* drain = q_free + 2;
  uint64_t* q_full = drain + 1;             // kTma: by segment % q_bufs
  uint64_t* edge = q_full + 2;              // kTma: V of units whose values are checked, in turn: arrived,
  uint64_t* checked = edge + kNotes;        // and checked
  uint64_t* pairs = checked + kNotes;       // of softmax warps that share rows, by tile and quarter
  Note* notes = reinterpret_cast<Note*>(smem + L::kNote);
  SegNote* seg_notes = reinterpret_cast<SegNote*>(smem + L::kSegNote);  // by segment & (kNotes - 1)
  volatile uint64_t* bad = reinterpret_cast<uint64_t*>(smem + L::kBad);
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  int64_t* s_total = reinterpret_cast<int64_t*>(misc + 2);
  const int q_tile = a.q_rows * DP * 2;     // bytes of a tile's Q
  const int q_odd = a.q_bufs - 1;           // 1: segments take turns with Q
  unsigned char* const q_smem = smem + kHead;
  unsigned char* const ring = q_smem + (a.q_bufs * kRows * q_tile + 1023) / 1024 * 1024;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform for the compiler, too

  if (tid < kNumBars) {
    const uint64_t* b = &bars[tid];
    int count = 1;
    if (b < empty) count = kTma ? 1 : kCopiers;
    if (b >= note_full && b < note_free) count = kTma ? 1 : kCopiers;
    if (b >= note_free && b < s_full) count = 1 + (kTma ? kReaders : 0);
    if (b >= p_full && b < o_full) count = a.warps;
    if (b >= o_free && b < q_free) count = kHalves * a.warps;
    if (b >= pairs) count = 2;
    mbar_init(&bars[tid], count);
    mbar_fence_init();
  }
  if (tid < kBadRing) bad[tid] = 0;
  if (tid == 0) *abort = 0;
  pdl_allow_next();
  pdl_wait();
  if (warp == kIssuer) tmem_alloc(tmem_ptr, 512);

  // ---- where the requests' units begin (by thread, in the ring's place)
  const int segs = a.kv_heads * a.passes, rounds = segs / a.gang;
  const int per = (a.num_reqs + kThreads - 1) / kThreads;
  int64_t* s_before = reinterpret_cast<int64_t*>(ring);   // [kThreads] units before each thread's requests
  int64_t* s_warp = s_before + kThreads;
  {
    const int r_lo = min(a.num_reqs, tid * per), r_hi = min(a.num_reqs, r_lo + per);
    uint32_t err = 0;
    int64_t mine = 0;
    for (int r = r_lo; r < r_hi; ++r) mine += (int64_t)request(a, r, err).units * rounds;
    if (blockIdx.x == 0) report(a.err, err);
    const int64_t incl = warp_inclusive_scan<int64_t>(mine);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    s_before[tid] = before;
    if (tid == kThreads - 1) *s_total = before + mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_ptr, 0);
  const int64_t total = *s_total;
  const int64_t share = (total + a.gangs - 1) / a.gangs;
  const int my_gang = blockIdx.x / a.gang, member = blockIdx.x - my_gang * a.gang;
  const int64_t begin = my_gang * share;
  const int64_t count = my_gang < a.gangs && begin < total ? min(share, total - begin) : 0;

  int64_t issued = 0, edges_used = 0;        // copying warps (kTma): units, of them through edge barriers
  auto wait = [&](uint64_t* b, uint32_t parity) { return role_wait(b, parity & 1, abort); };
  // A reader waits for its next note, reads what it wants of it and gives it back.
  auto note_there = [&](int64_t u) { return wait(&note_full[u & (kNotes - 1)], (uint32_t)(u >> 3)); };
  auto note_done = [&](int64_t u) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&note_free[u & (kNotes - 1)]);
  };

  // Values of the step's rows (key `step` on) that are not finite: 0, and their rows noted.
  auto check_values = [&](int y, int step, int seg_no, int s) {
    if (y < step) return;
    unsigned char* row = ring + s * L::kSlot + y * 128;
    bool any = false;
#pragma unroll 4
    for (int c = 0; c < kPieces; ++c) {
      uint4* p = reinterpret_cast<uint4*>(row + (c >> 3) * (kTile * 128) + (((c & 7) ^ (y & 7)) << 4));
      uint4 v = *p;
      uint32_t e[4] = {v.x, v.y, v.z, v.w};
      bool hit = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if ((e[k] & 0x7f80u) == 0x7f80u) e[k] &= 0xffff0000u, hit = true;
        if ((e[k] & 0x7f800000u) == 0x7f800000u) e[k] &= 0xffffu, hit = true;
      }
      if (hit) *p = make_uint4(e[0], e[1], e[2], e[3]);
      any |= hit;
    }
    if (any)
      atomicOr(reinterpret_cast<unsigned long long*>(smem + L::kBad) + seg_no, 1ull << (y - step));
  };
  if (warp >= kCopy) {
    // ---------------------------------------------------------------- copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    // TMA: 0 describes, 1 and 2 copy K and V, 3 loads Q, which has the least to do and shares the issuer's scheduler
    const int w = kTma && (warp - kCopy) % 3 == 0 ? 3 - (warp - kCopy) : warp - kCopy;
    uint32_t err = 0;
    if (w == 0 && lane == 0) a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);  // until it is known better
    // the first unit: the request whose units hold `begin`
    int r = 0, seg = 0, tile = 0;
    if (count > 0) {
      int lo = 0, hi = kThreads;  // last thread whose requests begin at or before it
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_before[mid] <= begin) lo = mid; else hi = mid;
      }
      r = lo * per;
      int64_t at = s_before[lo];
      uint32_t ignore = 0;
      int units = request(a, r, ignore).units;
      while (at + (int64_t)units * rounds <= begin) {
        at += (int64_t)units * rounds;
        units = request(a, ++r, ignore).units;
      }
      const int64_t rest = begin - at;
      seg = (int)(rest / units) * a.gang + member;
      tile = (int)(rest % units);
    }
    fence_proxy_async_smem();
    asm volatile("bar.sync 2, 128;" ::: "memory");  // before the ring is written
    const int sub = lane / kPieces, piece = lane % kPieces;
    constexpr int kPer = 32 / kPieces;      // rows of a copy instruction
    const bool piece_real = piece * 8 < a.head_dim;
    // Rows of Q of a segment, shared by `warps` warps of which this is number `me`.
    auto copy_q = [&](int first, int rows, int head, int pass, int buf, int me, int warps) {
      // from a row to this warp's next one: tokens and heads, and what that moves the source by
      const int ahead = warps * kPer, tok_step = ahead / a.group, g_step = ahead - tok_step * a.group;
      const int64_t move = tok_step * a.q_stride + (int64_t)g_step * a.head_dim;
      const int64_t wrap = a.q_stride - (int64_t)a.group * a.head_dim;  // a token more, a group of heads less
      for (int t = 0; t < kRows; ++t) {
        const int row0 = (pass * kRows + t) * kTile, left = min(rows * a.group - row0, kTile);  // rows of this tile
        int y = me * kPer + sub, g = row0 + y;
        const int tok = g / a.group;
        g -= tok * a.group;
        const __nv_bfloat16* src = a.q + (int64_t)(first + tok) * a.q_stride +
                                   (int64_t)(head * a.group + g) * a.head_dim + piece * 8;
        const uint32_t q_at = smem_addr(q_smem) + (buf * kRows + t) * q_tile + (piece >> 3) * (a.q_rows * 128);
#pragma unroll 4
        for (; y < left; y += ahead) {
          copy16(q_at + y * 128 + (((piece & 7) ^ (y & 7)) << 4), piece_real ? src : a.q, piece_real);
          g += g_step;
          src += move;
          if (g >= a.group) g -= a.group, src += wrap;
        }
      }
    };
    if (kTma && w == 3) {
      // -------------------------------------------------------------- Q
      // By TMA where a tile's rows are whole tokens; its rows behind the request's are of no use then.
      const bool leader = elect_one();
      if (leader && a.q_box > 0) tma_prefetch_map(&q_map);
      const int box_bytes = a.q_box * a.group * 128;
      int64_t segment = -1, loaded = 0;
      for (int64_t u = 0; u < count; ++u) {
        if (!note_there(u)) break;
        const int flags = notes[u & (kNotes - 1)].flags;
        if (flags & kFirst) ++segment;
        const SegNote g = seg_notes[segment & (kNotes - 1)];
        note_done(u);
        if (flags & kFirst) {
          if (segment >= a.q_bufs && !wait(&q_free[segment & q_odd], (uint32_t)(segment >> q_odd) - 1)) break;
          const int buf = (int)(segment & q_odd);
          if (a.q_box > 0) {
            if (leader) {
              const int tiles = kRows == 2 && (flags & kTwo) ? 2 : 1;
              mbar_arrive_expect_tx(&q_full[buf], tiles * (DP / 64) * box_bytes);
              for (int t = 0; t < tiles; ++t)
#pragma unroll
                for (int c = 0; c < DP / 64; ++c)
                  tma_load_3d(q_smem + (buf * kRows + t) * q_tile + c * (a.q_rows * 128), &q_map, 64 * c,
                              g.head * a.group, g.first + (g.pass * kRows + t) * a.q_box, &q_full[buf]);
            }
            __syncwarp();
            loaded = segment + 1;
          } else {
            copy_q(g.first, g.count, g.head, g.pass, buf, 0, 1);
            copy_commit();
            copy_wait<0>();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[buf]);
          }
        }
      }
      // none in flight when the shared memory goes to another CTA
      for (int64_t g = max((int64_t)0, loaded - a.q_bufs); g < loaded; ++g)
        mbar_wait_bounded(&q_full[g & q_odd], (uint32_t)(g >> q_odd) & 1);
    } else if (kTma && w > 0) {
      // -------------------------------------------------------------- copies of K (1) or V (2)
      const bool is_v = w == 2, leader = elect_one();
      const CUtensorMap* const map = is_v ? &v_map : &k_map;
      if (leader) tma_prefetch_map(map);
      const int boxes = kTile / a.box, box_bytes = a.box * 128;
      int slot = is_v ? 1 : 0;
      uint32_t turn = 0;
      for (int64_t u = 0; u < count; ++u) {
        if (!note_there(u)) break;
        const Note& n = notes[u & (kNotes - 1)];
        const int flags = n.flags, head = n.head, token = n.tokens[lane & 15];
        note_done(u);
        if (turn > 0 && !wait(&empty[slot], turn - 1)) break;
        const bool check = is_v && (flags & kEdge);
        uint64_t* const bar = check ? &edge[edges_used & (kNotes - 1)] : &full[slot];
        unsigned char* const to = ring + slot * L::kSlot;
        if (leader) {
          mbar_arrive_expect_tx(bar, L::kSlot);
          if (check) mbar_arrive(&full[slot]);  // its phases count the turns of the ring
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < boxes; ++i) {
          const int z = __shfl_sync(kFull, token, i);  // a box that is nowhere reads zeros
          if (leader) {
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
              tma_load_3d(to + c * (kTile * 128) + i * box_bytes, map, 64 * c, head, z, bar);
          }
        }
        edges_used += check;
        ++issued;
        slot += 2;
        if (slot >= a.slots) slot -= a.slots, ++turn;
      }
    } else {
      // -------------------------------------------------------------- units, in order
      // 32 requests at a time, one a lane
      int base = r;
      Req mine = {};
      auto look = [&]() {
        uint32_t ignore = 0;
        mine = Req{0, 0, 0, 0, 0, 0, 0};
        if (base + lane < a.num_reqs) mine = request(a, base + lane, ignore);
      };
      Req now = {};
      // of the unit: where it is in the request, its first position and table row
      uint32_t pos = 0;
      const int32_t* row = nullptr;
      auto take = [&]() {
        now.first = __shfl_sync(kFull, mine.first, r - base);
        now.count = __shfl_sync(kFull, mine.count, r - base);
        now.lo = __shfl_sync(kFull, mine.lo, r - base);
        now.hi = __shfl_sync(kFull, mine.hi, r - base);
        now.ctx = __shfl_sync(kFull, mine.ctx, r - base);
        now.base = __shfl_sync(kFull, mine.base, r - base);
        now.units = __shfl_sync(kFull, mine.units, r - base);
        row = a.table + (int64_t)r * a.stride;
      };
      // This lane's row (kTma: box) of a unit, in two steps, so that its table entry arrives while the
      // unit before it is dealt with: block and offset, then the token in the pool (kNowhere: none).
      constexpr uint32_t kNowhere = ~0u;
      const int boxes = kTile / a.box;
      const uint32_t lane_at = kTma ? lane * a.box : w * 32 + lane;
      const uint32_t T = (uint32_t)a.div.size;
      int32_t next_block = kNull;
      uint32_t next_off = 0;
      auto look_up = [&]() {
        const uint32_t p = pos + lane_at;
        next_block = kNull;
        if (p < now.hi && (!kTma || lane < boxes)) {
          const uint32_t lb = a.div.shift >= 0 ? p >> a.div.shift : p / T;
          next_off = p - lb * T;
          next_block = row[lb];
        }
      };
      auto token = [&]() {
        if (next_block == kNull) return kNowhere;
        if (next_block < 0 || next_block >= a.num_blocks) {
          err |= KV_ERR_BAD_BLOCK;
          return kNowhere;
        }
        return (uint32_t)next_block * T + next_off;
      };
      if (count > 0) {
        look();
        take();
        pos = now.base + (uint32_t)tile * kTile;
        look_up();
      }
      constexpr int kTurns = 8 / kPer;        // copy instructions after which the swizzle repeats
      const bool dense = a.head_dim == DP;
      const uint32_t row_bytes = (uint32_t)(a.kv_heads * a.head_dim * 2);
      const char* const k_lane = reinterpret_cast<const char*>(a.k_cache) + (piece_real ? piece * 16 : 0);
      const int64_t k_to_v = reinterpret_cast<const char*>(a.v_cache) - reinterpret_cast<const char*>(a.k_cache);
      // rows w * 32 + i * kPer + sub: their 8-row groups are 1024 bytes, column blocks of 64 channels apart
      uint32_t dst_lane[kTurns];
#pragma unroll
      for (int i = 0; i < kTurns; ++i)
        dst_lane[i] = smem_addr(ring) + (uint32_t)((w * 32 + i * kPer + sub) * 128 + (piece >> 3) * (kTile * 128) +
                                                   (((piece & 7) ^ (i * kPer + sub)) << 4));

      int64_t told = 0;         // units that the issuer may use
      int k_slot = 0, v_slot = 1, told_slot = 0;
      uint32_t k_turn = 0, v_turn = 0;
      int64_t segment = -1;     // of this CTA, counted
      int hist_step[kLag + 2], hist_seg[kLag + 2];  // of the last units: where the step's rows begin
#pragma unroll
      for (int i = 0; i < kLag + 2; ++i) hist_step[i] = kTile, hist_seg[i] = 0;
      bool ok = true;
      // Unit `told` has arrived: the issuer may use it.  `back`: units issued behind it.
      auto tell = [&](int back) {
        const int s0 = told_slot, s1 = s0 + 1 == a.slots ? 0 : s0 + 1;
        int step = kTile, seg_no = 0;
#pragma unroll
        for (int i = 0; i < kLag + 2; ++i)
          if (i == back) step = hist_step[i], seg_no = hist_seg[i];
        if (step < kTile) {
          __syncwarp();
          check_values(w * 32 + lane, step, seg_no, s1);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[s0]);
          mbar_arrive(&full[s1]);
        }
        ++told;
        told_slot = s1 + 1 == a.slots ? 0 : s1 + 1;
      };
      // The issuer may need units in flight to get to the end of a wait of this role: the oldest ones
      // are told about until it is over.  `so_far`: units whose copies are under way or done.
      auto wait_telling = [&](uint64_t* b, uint32_t parity, int64_t so_far) {
        while (told < so_far && !__any_sync(kFull, mbar_try_wait(b, parity & 1))) {
          const int back = (int)(so_far - 1 - told);  // groups behind the oldest, kLag at most
          if (back == 0) copy_wait<0>();
          else if (back == 1) copy_wait<1>();
          else if (back == 2) copy_wait<2>();
          else copy_wait<3>();
          tell(back + 1);  // the next unit is in the history already
        }
        return wait(b, parity);
      };
      int head = seg / a.passes;
      for (int64_t u = 0; ok && u < count; ++u) {
        // this unit
        const uint32_t here = token();
        const bool first = u == 0 || tile == 0, from_start = tile == 0;
        const bool to_end = tile + 1 == now.units, last = to_end || u + 1 == count;
        const int step = max(-kTile, min(kTile, (int)(now.ctx - pos)));
        const int lo = from_start ? (int)(now.lo - pos) : 0;  // its keys [lo, hi) are positions of the request
        const int hi = (int)min((uint32_t)kTile, now.hi - pos);
        const Req req = now;
        const int here_r = r, here_head = head, here_pass = seg - head * a.passes;
        if (last && !to_end) {  // a segment that begins here and ends with another CTA: how far the join reaches
          const int64_t from = begin + u - tile;  // the segment's first unit
          if (w == 0 && lane == 0 && from >= begin)
            a.joins[blockIdx.x] = make_int4(r, seg, (int)((from + now.units - 1) / share), now.count);
        }
        // the next one, and its table entries
        if (u + 1 < count) {
          pos += kTile;
          if (++tile == now.units) {
            tile = 0;
            seg += a.gang;
            if (seg >= segs) {
              seg = member;
              do {
                if (++r >= base + 32) {
                  base = r;
                  look();
                }
              } while (__shfl_sync(kFull, mine.units, r - base) == 0);
              take();
            }
            head = seg / a.passes;
            pos = now.base;
          }
          look_up();
        }
        if (first) ++segment;
        if constexpr (!kTma) {
#pragma unroll
          for (int i = kLag + 1; i > 0; --i) hist_step[i] = hist_step[i - 1], hist_seg[i] = hist_seg[i - 1];
          hist_step[0] = step;
          hist_seg[0] = (int)(segment & (kBadRing - 1));
        }
        // describe it
        if (u >= kNotes) ok = wait(&note_free[u & (kNotes - 1)], (uint32_t)(u >> 3) - 1);
        if (!ok) break;
        uint32_t valid = __ballot_sync(kFull, here != kNowhere);
        Note& n = notes[u & (kNotes - 1)];
        if constexpr (kTma) {
          if (lane < boxes) n.tokens[lane] = here == kNowhere ? -a.box : (int)here;
          // word `lane`: its boxes' bits, spread over their keys
          uint32_t word = 0;
          if (a.box >= 32) {
            if ((valid >> (32 * lane / a.box & 31)) & 1u) word = kFull;
          } else {
            const int some = 32 / a.box;
            const uint32_t ones = (1u << a.box) - 1u;
            valid >>= lane * some & 31;
            word = (valid & 1u ? ones : 0u) | (valid & 2u ? ones << a.box : 0u);
            if (some == 4) word |= (valid & 4u ? ones << 16 : 0u) | (valid & 8u ? ones << 24 : 0u);
          }
          const int from = lo - 32 * lane, to = hi - 32 * lane;
          if (from > 0) word &= from < 32 ? kFull << from : 0u;
          if (to < 32) word &= to > 0 ? (1u << to) - 1u : 0u;
          if (lane < 4) n.valid[lane] = word;
        } else if (lane == 0) {
          n.valid[w] = valid;
        }
        if (w == 0 && lane == 0) {
          n.step = step;
          n.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (to_end ? kToEnd : 0) |
                    (first && from_start ? kFromStart : 0) |
                    (kTma && (step < kTile || lo > 0 || hi % a.box != 0) ? kEdge : 0) |
                    (req.count * a.group > (here_pass * kRows + 1) * kTile ? kTwo : 0);
          n.head = here_head;
          n.seen = lo | hi << 8;
          if (first) {
            SegNote& g = seg_notes[segment & (kNotes - 1)];
            g.r = here_r;
            g.head = here_head;
            g.pass = here_pass;
            g.first = req.first;
            g.count = req.count;
            g.ctx = req.ctx;
            bad[(segment + 7) & (kBadRing - 1)] = 0;  // all have read that one, none written
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&note_full[u & (kNotes - 1)]);
        if constexpr (kTma) continue;
        // copy it
        if (first && segment >= a.q_bufs)
          ok = wait_telling(&q_free[segment & q_odd], (uint32_t)(segment >> q_odd) - 1, u);
        ok = ok && (k_turn == 0 || role_wait(&empty[k_slot], (k_turn - 1) & 1, abort)) &&
             (v_turn == 0 || role_wait(&empty[v_slot], (v_turn - 1) & 1, abort));
        if (!ok) break;
        if (first)  // Q with the segment's first unit
          copy_q(req.first, req.count, here_head, here_pass, (int)(segment & q_odd), w, kCopiers);
        const char* const src = k_lane + here_head * a.head_dim * 2;
        const uint32_t k_to = k_slot * L::kSlot, v_to = v_slot * L::kSlot;
        if (valid == kFull && dense) {
#pragma unroll
          for (int i = 0; i < 32 / kPer; ++i) {
            const char* p = src + (uint64_t)__shfl_sync(kFull, here, i * kPer + sub) * row_bytes;
            const uint32_t to = dst_lane[i % kTurns] + (i / kTurns) * 1024;
            copy16(to + k_to, p);
            copy16(to + v_to, p + k_to_v);
          }
        } else {
#pragma unroll 4
          for (int i = 0; i < 32 / kPer; ++i) {
            const uint32_t x = __shfl_sync(kFull, here, i * kPer + sub);
            const bool real = x != kNowhere && piece_real;
            const char* p = real ? src + (uint64_t)x * row_bytes : src;
            const uint32_t to = dst_lane[i % kTurns] + (i / kTurns) * 1024;
            copy16(to + k_to, p, real);
            copy16(to + v_to, p + k_to_v, real);
          }
        }
        copy_commit();
        k_slot += 2;
        if (k_slot >= a.slots) k_slot -= a.slots, ++k_turn;
        v_slot += 2;
        if (v_slot >= a.slots) v_slot -= a.slots, ++v_turn;
        if (u - told >= kLag) {
          copy_wait<kLag>();
          tell((int)(u - told));
        }
      }
      if constexpr (!kTma) {
        copy_wait<0>();
        while (ok && told < count) tell((int)(count - 1 - told));
      }
    }
    report(a.err, err);
  } else if (warp >= kIssuer) {
    // ---------------------------------------------------------------- matrix instructions
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));  // the whole warpgroup
    if (warp == kIssuer) {
      constexpr uint32_t s_desc = mma_desc(128, kTile, false), o_desc = mma_desc(128, DP, true);
      const uint32_t ring_at = smem_addr(ring), q_base = smem_addr(q_smem);
      const bool leader = elect_one();
      const uint32_t q_cols = (uint32_t)(a.q_rows * 128) >> 4;  // from a 64-channel block of Q to the next
      auto scores = [&](uint32_t d, uint32_t q_at, int slot) {
        const uint64_t qd = smem_desc(q_at, 16), kd = smem_desc(ring_at + slot * L::kSlot, 16);
        if (leader) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(d, qd + (k / 4) * q_cols + (k % 4) * 2, kd + (((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4),
                   s_desc, k > 0);
        }
        __syncwarp();
      };
      auto values = [&](uint32_t d, uint32_t p, int slot, bool add, int half) {
        const uint64_t vd = smem_desc(ring_at + slot * L::kSlot, kTile * 128) + half * ((kTile / 2 * 128) >> 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_ts(d, p + half * (kTile / 2) + k * 8, vd + k * (2048 >> 4), o_desc, add || k > 0);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* b) {
        if (leader) mma_commit(b);
        __syncwarp();
      };
      bool ok = true;
      int slot = 0;
      uint32_t turn = 0;
      auto step = [&]() {
        if (++slot == a.slots) {
          slot = 0;
          ++turn;
        }
      };
      int64_t segment = -1, edges = 0;
      // V of a unit, through the warp that checks it where it has values to check
      auto values_there = [&](uint64_t* b, uint32_t parity, bool check) {
        if (!kTma || !check) return wait(b, parity);
        ++edges;
        return wait(&checked[(edges - 1) & (kNotes - 1)], (uint32_t)((edges - 1) >> 3));
      };
      // the first unit's flags, the next ones' ahead of time
      int flags = 0;
      auto read_flags = [&](int64_t u) {
        if (!wait(&note_full[u & (kNotes - 1)], (uint32_t)(u >> 3))) return false;
        flags = notes[u & (kNotes - 1)].flags;
        return true;
      };
      // all have read a unit's note once its weights are there
      auto give_back = [&](int64_t u) {
        if (leader) mbar_arrive(&note_free[u & (kNotes - 1)]);
        __syncwarp();
      };
      if (count > 0) ok = read_flags(0);
      if constexpr (kRows == 1) {
        // unit u's scores, then unit u - 1's products with V; behind a segment's end the products first, as
        // the next one's Q may be late
        int v_slot = 0, v_flags = 0;
        uint32_t v_turn = 0;
        int64_t v_segment = 0;
        auto products = [&](int64_t u) {
          const uint32_t d = tmem + 2 * kTile + (uint32_t)(v_segment & 1) * DP, p = tmem + (uint32_t)(u & 1) * kTile;
          const bool first = v_flags & kFirst;
          if (first && v_segment >= 2 && !wait(&o_free[v_segment & 1], (uint32_t)(v_segment >> 1) - 1)) return false;
          if (!values_there(&full[v_slot], v_turn, v_flags & kEdge) || !wait(&p_full[2 * (u & 1)], (uint32_t)(u >> 1)))
            return false;
          tc_fence_after();
          values(d, p, v_slot, !first, 0);
          if (!wait(&p_full[2 * (u & 1) + 1], (uint32_t)(u >> 1))) return false;
          tc_fence_after();
          values(d, p, v_slot, true, 1);
          commit(&o_full[0]);
          commit(&empty[v_slot]);
          give_back(u);
          return true;
        };
        for (int64_t u = 0; ok && u <= count; ++u) {
          const bool more = u < count, first = more && (flags & kFirst);
          if (first) ++segment;
          // each of the two once in the code
#pragma unroll 1
          for (int part = 0; ok && part < 2; ++part) {
            if ((part == 1) == first) {
              if (!more) continue;
              ok = wait(&full[slot], turn) &&
                   (!kTma || !first || wait(&q_full[segment & q_odd], (uint32_t)(segment >> q_odd)));
              if (!ok) break;
              tc_fence_after();
              scores(tmem + (uint32_t)(u & 1) * kTile, q_base + (uint32_t)(segment & q_odd) * q_tile, slot);
              commit(&s_full[u & 1]);
              commit(&empty[slot]);
              if (flags & kLast) commit(&q_free[segment & q_odd]);
            } else if (u > 0) {
              ok = products(u - 1);
            }
          }
          step();
          v_slot = slot;
          v_turn = turn;
          v_segment = segment;
          v_flags = flags;
          step();
          if (ok && u + 1 < count) ok = read_flags(u + 1);
        }
      } else {
        // The tiles take turns: P V of a tile, then its next scores behind it.  A tile without rows in this
        // segment goes through the same waits with no instruction.
        uint32_t segments = 0;   // ended
        int v_slot = 0;
        auto tile_scores = [&](int t, bool two) {
          if (t == 0 || two)
            scores(tmem + t * kTile, q_base + ((uint32_t)(segment & q_odd) * 2 + t) * q_tile, slot);
          commit(&s_full[t]);
        };
        auto scores_done = [&]() {  // of the unit whose flags these are
          commit(&empty[slot]);
          if (flags & kLast) commit(&q_free[segment & q_odd]);
          step();
        };
        auto first_scores = [&]() {  // of a segment's first unit here
          ++segment;
          if (!wait(&full[slot], turn) ||
              (kTma && !wait(&q_full[segment & q_odd], (uint32_t)(segment >> q_odd))))
            return false;
          tc_fence_after();
#pragma unroll 1
          for (int t = 0; t < 2; ++t) tile_scores(t, flags & kTwo);
          scores_done();
          return true;
        };
        if (count > 0) ok = ok && first_scores();
        for (int64_t u = 0; ok && u < count; ++u) {
          v_slot = slot;         // V of this unit
          const uint32_t v_turn = turn;
          const int now = flags;
          const bool first = now & kFirst, last = now & kLast, two = now & kTwo;
          step();
          ok = values_there(&full[v_slot], v_turn, now & kEdge) && (u + 1 == count || read_flags(u + 1)) &&
               (last || wait(&full[slot], turn));
#pragma unroll 1
          for (int t = 0; ok && t < 2; ++t) {
            const uint32_t d = tmem + 2 * kTile + t * DP, p = tmem + t * kTile;
            ok = (!first || segments == 0 || wait(&o_free[t], segments - 1)) && wait(&p_full[2 * t], (uint32_t)u);
            if (!ok) break;
            tc_fence_after();
            if (t == 0 || two) values(d, p, v_slot, !first, 0);
            ok = wait(&p_full[2 * t + 1], (uint32_t)u);
            if (!ok) break;
            tc_fence_after();
            if (t == 0 || two) values(d, p, v_slot, true, 1);
            if (!last) tile_scores(t, two);
            else commit(&o_full[t]);
          }
          if (ok) {
            commit(&empty[v_slot]);
            give_back(u);
            if (!last) {
              scores_done();
            } else {
              ++segments;
              if (u + 1 < count) ok = first_scores();
            }
          }
        }
      }
      // none of the matrix unit's arrivals may come after the shared memory has gone to another CTA
      __syncwarp();
      if (leader) mma_commit(drain);
      mbar_wait_bounded(drain, 0);
    } else if (kTma && warp == kIssuer + 1) {
      // -------------------------------------------------------------- values at the edges
      int64_t segment = -1, edges = 0;
      int slot = 1;              // V of the unit
      for (int64_t u = 0; u < count; ++u) {
        if (!note_there(u)) break;
        const Note& n = notes[u & (kNotes - 1)];
        const int flags = n.flags, step = n.step, from = n.seen & 255, to = n.seen >> 8;
        note_done(u);
        if (flags & kFirst) ++segment;
        if (flags & kEdge) {
          if (!wait(&edge[edges & (kNotes - 1)], (uint32_t)(edges >> 3))) break;
          for (int y = lane; y < kTile; y += 32) {
            if (y < from || y >= to) {  // of the block, but not of the request
#pragma unroll
              for (int c = 0; c < kPieces; ++c)
                *reinterpret_cast<uint4*>(ring + slot * L::kSlot + (c >> 3) * (kTile * 128) + y * 128 +
                                          (((c & 7) ^ (y & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            } else {
              check_values(y, step, (int)(segment & (kBadRing - 1)), slot);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&checked[edges & (kNotes - 1)]);
          ++edges;
        }
        slot += 2;
        if (slot >= a.slots) slot -= a.slots;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // requests without a position: zeros
    const int64_t vecs = (int64_t)a.q_heads * a.head_dim / 8;
    for (int r = blockIdx.x; r < a.num_reqs; r += gridDim.x) {
      uint32_t ignore = 0;
      const Req q = request(a, r, ignore);
      if (q.units > 0 || q.count <= 0) continue;
      uint4* o = reinterpret_cast<uint4*>(a.out) + q.first * vecs;
      for (int64_t i = tid; i < q.count * vecs; i += 128 * kRows * kHalves) o[i] = make_uint4(0, 0, 0, 0);
    }
    // With two tiles, two warps share 32 rows: each takes half of a unit's keys, and half of O's channels.
    const int t = kHalves == 2 ? warp >> 3 : 0, half = kHalves == 2 ? (warp >> 2) & 1 : 0, quarter = warp & 3;
    constexpr int kKeys = kTile / kHalves, kChannels = DP / kHalves;
    constexpr int kLook = kRows == 1 ? 64 : 32, kChunk = 32;  // keys in registers at a time
    if (quarter < a.warps) {
      // -------------------------------------------------------------- softmax
      const uint32_t lanes = (uint32_t)quarter << 21;     // this warp's 32 lanes, in bits 16..
      const float c = a.scale_log2;
      const int in_tile = quarter * 32 + lane;
      uint64_t* const pair_bar = &pairs[t * 4 + quarter];
      float* const top_at = reinterpret_cast<float*>(smem + L::kTops) + t * kTile + in_tile;
      uint32_t* const words = reinterpret_cast<uint32_t*>(smem + L::kWords) + (t * 4 + quarter) * 2;
      uint32_t meets = 0;
      auto meet = [&]() {  // with the other warp of these rows
        __syncwarp();
        if (lane == 0) mbar_arrive(pair_bar);
        return wait(pair_bar, meets++);
      };
      // what `both` makes of the two warps' values, in both
      auto join = [&](float& x, auto both) {
        if (kHalves == 1) return true;
        if (half == 0) *top_at = x;
        if (!meet()) return false;
        if (half == 1) *top_at = x = both(*top_at, x);
        if (!meet()) return false;
        if (half == 0) x = *top_at;
        return true;
      };
      int64_t segment = -1;
      uint32_t segments = 0;                 // of this tile
      float ref = 0.f;
      uint64_t part[2] = {0, 0};             // sums of this warp's weights, two by two
      uint64_t mask = 0;
      int tok = 0, g = 0;
      bool mine = false, from_start = false;
      bool ok = true;
      SegNote g_note = {};
      for (int64_t u = 0; u < count; ++u) {
        const int sb = kRows == 1 ? (int)(u & 1) : t;
        ok = wait(&s_full[sb], (uint32_t)(kRows == 1 ? u >> 1 : u));
        if (!ok) break;
        tc_fence_after();
        // the issuer has read the note that this unit's scores came behind
        const Note& n = notes[u & (kNotes - 1)];
        const int flags = n.flags, step = n.step;
        uint32_t all_valid = kFull;
#pragma unroll
        for (int b = 0; b < kKeys / 32; ++b) all_valid &= n.valid[half * (kKeys / 32) + b];
        if (flags & kFirst) {
          ++segment;
          g_note = seg_notes[segment & (kNotes - 1)];
          const int row = (g_note.pass * kRows + t) * kTile + in_tile;
          tok = row / a.group;
          g = row - tok * a.group;
          mine = tok < g_note.count;
          from_start = flags & kFromStart;
          mask = 0;
          if (mine) mask = a.tree_mask != nullptr ? (uint64_t)a.tree_mask[g_note.first + tok] : ~0ull >> (63 - tok);
        }
        if (kRows == 2 && t == 1 && !(flags & kTwo)) {  // no rows here
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * sb + half]);
          if (flags & kLast) {
            ok = wait(&o_full[t], segments);
            if (!ok) break;
            ++segments;
            if (lane == 0) mbar_arrive(&o_free[t]);
          }
          continue;
        }
        const uint32_t s_at = tmem + lanes + sb * kTile + half * kKeys;
        const uint32_t o_at = tmem + lanes + 2 * kTile + (kRows == 1 ? (uint32_t)(segment & 1) : (uint32_t)t) * DP +
                              half * kChannels;
        // kLook and kChunk keys at a time, in loops: the code of a whole tile, unrolled, has the four schedulers
        // wait for instructions (twice the time with four warps as with one).  64 trees of 2 to 25 rows: 126.6 us
        // with 64 keys' weights at a time, 124.5 with 32, 123 with the maxima of 64 then; one row and heads of 64
        // channels, where a warp is alone with its latency, 210, 239 and 229.
        // Hidden logits first, in a loop of their own: few units have any.
        if (step < kTile || all_valid != kFull) {
#pragma unroll 1
          for (int b = 0; b < kKeys / 32; ++b) {
            // what this row sees of these keys: the context before `step`, its mask from there on
            const int from = step - kKeys * half - 32 * b;
            uint32_t see = from >= 32 ? kFull : from > 0 ? (1u << from) - 1u : 0u;
            if (from > 0) see |= from < 32 ? (uint32_t)(mask << from) : 0u;
            else see |= from > -64 ? (uint32_t)(mask >> -from) : 0u;
            see &= n.valid[half * (kKeys / 32) + b];
            uint32_t s[32];
            tmem_ld32(s_at + 32 * b, s);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!((see >> y) & 1u)) s[y] = 0xff800000u;
            tmem_st32(s_at + 32 * b, s);
            tmem_wait_st();
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int b = 0; b < kKeys / kLook; ++b) {
          uint32_t s[kLook];
#pragma unroll
          for (int i = 0; i < kLook / 32; ++i) tmem_ld32(s_at + kLook * b + 32 * i, s + 32 * i);
          tmem_wait_ld();
#pragma unroll
          for (int z = 0; z < kLook; z += 4)
#pragma unroll
            for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], __uint_as_float(s[z + y]));
        }
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        // One tile: the last unit's P V may still run (S of this one came behind the one before that; two
        // tiles: behind the last one).  A barrier tells its last phase from the one before and no
        // further, so it is looked at before this warp lets this unit's P V run: for the rescale,
        // and ahead of the output's own wait.
        if (kRows == 1 && u > 0 && (flags & kLast)) {
          ok = wait(&o_full[0], (uint32_t)u - 1);
          if (!ok) break;
          tc_fence_after();
        }
        // does a row's maximum pass the reference, here or in the other warp?
        bool rise = flags & kFirst;
        if (!rise) {
          const uint32_t word = __ballot_sync(kFull, mine && top > ref + kLazy);
          rise = word != 0;
          if (kHalves == 2) {
            uint32_t* const at = words + (u & 1) * 16;
            if (lane == 0) at[half] = word;
            ok = meet();
            if (!ok) break;
            rise |= *(volatile uint32_t*)&at[half ^ 1] != 0;
          }
        }
        if (rise) {
          ok = join(top, [](float x, float y) { return fmaxf(x, y); });
          if (!ok) break;
          if (flags & kFirst) {
            ref = top > -INFINITY ? top : kRefStart;
            part[0] = part[1] = 0;
          } else {
            if (kRows == 1 && !(flags & kLast)) {
              ok = wait(&o_full[0], (uint32_t)u - 1);
              if (!ok) break;
              tc_fence_after();
            }
            const bool raise = mine && top > ref + kLazy;
            const float f = raise ? ex2(ref - top) : 1.f;
            if (raise) ref = top;
            part[0] = mul2(part[0], pair(f, f));
            part[1] = mul2(part[1], pair(f, f));
#pragma unroll 1
            for (int b = 0; b < kChannels / 32; ++b) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * b, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32(o_at + 32 * b, o);
            }
          }
        }
        const uint64_t c2 = pair(c, c), r2 = pair(-ref, -ref);
#pragma unroll 1
        for (int b = 0; b < kKeys / kChunk; ++b) {
          uint32_t s[kChunk], p[kChunk / 2];
#pragma unroll
          for (int i = 0; i < kChunk / 32; ++i) tmem_ld32(s_at + kChunk * b + 32 * i, s + 32 * i);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < kChunk / 2; ++y) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])), c2, r2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            part[y & 1] = add2(part[y & 1], pair(e0, e1));
            p[y] = pack_bf16(e0, e1);
          }
          // over logits of the same 64 keys that are used up
          tmem_st16(s_at + (b >> 1) * 64 + (b & 1) * 16, p);
          if (b & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * sb + (kHalves == 2 ? half : b >> 1)]);
          }
        }
        if (!(flags & kLast)) continue;
        // ------------------------------------------------------------ output
        float sum;
        {
          float a0, a1, b0, b1;
          unpair(part[0], a0, a1);
          unpair(part[1], b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        }
        ok = join(sum, [](float x, float y) { return x + y; }) &&
             wait(&o_full[kRows == 1 ? 0 : t], kRows == 1 ? (uint32_t)u : segments);
        if (!ok) break;
        ++segments;
        tc_fence_after();
        const bool whole = from_start && (flags & kToEnd);
        uint64_t spoilt = bad[segment & (kBadRing - 1)];
        spoilt &= mask;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int in_part = t * kTile + in_tile;
        float* part_at = a.parts + ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * a.part_rows * DP;
        // 4 lanes hold 4 rows; they exchange 16-byte pieces, so that a store writes 64 bytes of
        // each of 8 rows
        const int64_t own = !mine ? -1
                            : whole ? ((int64_t)(g_note.first + tok) * a.q_heads + g_note.head * a.group + g) * a.head_dim
                                    : (int64_t)in_part * DP;
        int64_t to[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) to[y] = __shfl_sync(kFull, own, (lane & 28) + y);
#pragma unroll 1
        for (int b = 0; b < kChannels / 32; ++b) {
          const int col = half * kChannels + 32 * b;
          uint32_t o[32];
          tmem_ld32(o_at + 32 * b, o);
          tmem_wait_ld();
          // values that were set to 0, where this row sees them
          for (uint64_t left = spoilt; left != 0; left &= left - 1) {
            const int64_t p = (int64_t)g_note.ctx + __ffsll((long long)left) - 1;
            int64_t lb, off;
            a.div.divmod(p, lb, off);
            const int64_t blk = a.table[(int64_t)g_note.r * a.stride + lb];
            const __nv_bfloat16* v = a.v_cache + ((blk * a.div.size + off) * a.kv_heads + g_note.head) * a.head_dim;
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (col + y < a.head_dim && (__bfloat16_as_ushort(v[col + y]) & 0x7f80u) == 0x7f80u)
                o[y] = __float_as_uint(__uint_as_float(o[y]) + __bfloat162float(v[col + y]));
          }
          if (whole) {
            uint4 z[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t* e = o + 8 * y;
              auto two = [&](int k) {
                return pack_bf16(__uint_as_float(e[k]) * inv, __uint_as_float(e[k + 1]) * inv);
              };
              z[y] = make_uint4(two(0), two(2), two(4), two(6));
            }
            exchange(z[0], z[1], lane & 1, 1);
            exchange(z[2], z[3], lane & 1, 1);
            exchange(z[0], z[2], lane & 2, 2);
            exchange(z[1], z[3], lane & 2, 2);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (to[y] >= 0 && col + 8 * (lane & 3) < a.head_dim)
                *reinterpret_cast<uint4*>(a.out + to[y] + col + 8 * (lane & 3)) = z[y];
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 z[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                z[y] = make_uint4(o[16 * h + 4 * y], o[16 * h + 4 * y + 1], o[16 * h + 4 * y + 2], o[16 * h + 4 * y + 3]);
              exchange(z[0], z[1], lane & 1, 1);
              exchange(z[2], z[3], lane & 1, 1);
              exchange(z[0], z[2], lane & 2, 2);
              exchange(z[1], z[3], lane & 2, 2);
#pragma unroll
              for (int y = 0; y < 4; ++y)
                if (to[y] >= 0)
                  *reinterpret_cast<uint4*>(part_at + to[y] + col + 16 * h + 4 * (lane & 3)) = z[y];
            }
          }
        }
        if (!whole && mine && half == 0)
          reinterpret_cast<float2*>(a.parts + (int64_t)gridDim.x * 2 * a.part_rows * DP)[
              ((int64_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * a.part_rows + in_part] = make_float2(ref, sum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[kRows == 1 ? (int)(segment & 1) : t]);
      }
    }
  }
  // all roles have come so far: no matrix instruction or arrival is left, and no copy unless a wait ran out
  const bool copies = kTma && (warp == kCopy + 1 || warp == kCopy + 2);
  int64_t* const s_issued = reinterpret_cast<int64_t*>(smem + L::kTops);  // of K, of V
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (kTma && *abort != 0) {
    // this warp's copies in flight end before the shared memory goes to another CTA
    const int is_v = warp == kCopy + 2;
    if (copies && lane == 0) s_issued[is_v] = issued;
    __syncthreads();
    if (copies) {
      for (int64_t u = max((int64_t)0, issued - (a.slots + 1) / 2); u < issued; ++u) {
        // a slot whose next turn has begun was read, and its barrier may be a phase further
        const int64_t at = 2 * u + is_v, next = at + a.slots;
        if (next / 2 >= s_issued[next & 1]) mbar_wait_bounded(&full[at % a.slots], (uint32_t)(at / a.slots) & 1);
      }
      for (int64_t e = max((int64_t)0, edges_used - 6); e < edges_used; ++e)
        mbar_wait_bounded(&edge[e & (kNotes - 1)], (uint32_t)(e >> 3) & 1);
    }
  }
  if (warp == kIssuer) {
    tmem_dealloc(tmem, 512);
    if (lane == 0 && *abort != 0 && a.err != nullptr) atomicOr(a.err, KV_ERR_TIMEOUT);
  }
}

// Join: out = sum_i f_i o_i / sum_i f_i l_i, f_i = 2^(ref_i - max ref), over the parts of the
// segment that CTA x began and did not end: its own second part, then the first parts of the
// same member of the gangs behind it.  A thread has 4 channels, DP / 4 of them a row.  Every CTA looks
// through the list of such segments, so that their rows are shared out whoever began them: a row to a
// group, or, where there are fewer rows than CTAs, to all groups of a CTA, which take parts in turn.
// (With the rows of a segment left to blocks of the CTA that began it: one request of 8 rows behind
// 1001 tokens 18.6 us with the attention, 14.5 so; two of up to 109306 tokens, one KV head, 118 rows of 150
// parts, 57.6 and 28.1; 256 decode contexts 353 and 351; calls without a segment to join 0.5 more.  4 CTAs
// to one of the attention, 8 or 12: 64 trees 125, 122 and 120 us, calls without a join 0.4 apart.)
template <int DP, int kRows>
__global__ void __launch_bounds__(kJoinThreads) join_tree_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kWarps = kJoinThreads / 32, kLanes = DP / 4, kGroups = kJoinThreads / kLanes, kBatch = 4;
  __shared__ int4 s_join[kMaxCtas];
  __shared__ int s_end[kMaxCtas];            // rows to join of the segments that CTAs 0 .. x began
  __shared__ int s_sum[2 * kWarps];
  __shared__ float4 s_o[kGroups][kLanes];
  __shared__ float2 s_stat[kGroups];
  pdl_allow_next();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, ctas = a.gangs * a.gang;
  int end[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int x = h * kJoinThreads + tid;
    const int4 j = x < ctas ? a.joins[x] : make_int4(-1, 0, 0, 0);
    s_join[x] = j;
    end[h] = j.x < 0 ? 0 : max(0, min(j.w * a.group - j.y % a.passes * kRows * kTile, kRows * kTile));
  }
  if (!__syncthreads_or(end[0] | end[1])) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    end[h] = warp_inclusive_scan<int>(end[h]);
    if ((tid & 31) == 31) s_sum[h * kWarps + warp] = end[h];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int w = 0; w < 2 * kWarps; ++w)
      if (w < h * kWarps + warp) end[h] += s_sum[w];
    s_end[h * kJoinThreads + tid] = end[h];
  }
  __syncthreads();
  const int total = s_end[kMaxCtas - 1], group = tid / kLanes, lane = tid % kLanes;
  const bool together = total <= (int)gridDim.x;
  const int step = together ? kGroups : 1, sub = together ? group : 0;   // parts of this group
  const float2* stats = reinterpret_cast<const float2*>(a.parts + (int64_t)ctas * 2 * a.part_rows * DP);
  for (int item = together ? blockIdx.x : blockIdx.x * kGroups + group; item < total;
       item += gridDim.x * (kGroups / step)) {
    int x = 0;                               // the first one with item < s_end[x]
    for (int hi = kMaxCtas - 1; x < hi;) {
      const int mid = (x + hi) >> 1;
      if (s_end[mid] > item) hi = mid; else x = mid + 1;
    }
    const int row = item - (x > 0 ? s_end[x - 1] : 0);
    const int4 j = s_join[x];
    const int first = a.q_start[j.x];
    const int head = j.y / a.passes, pass = j.y - head * a.passes, row0 = pass * kRows * kTile;
    const int g0 = x / a.gang, member = x - g0 * a.gang;
    float top = kRefStart, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float2 (&st)[kBatch], const float4 (&v)[kBatch]) {
      float up = top;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) up = fmaxf(up, st[b].x);
      const float f = ex2(top - up);
      top = up;
      l *= f;
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float h = ex2(st[b].x - up);
        l = fmaf(st[b].y, h, l);
        o = make_float4(fmaf(v[b].x, h, o.x), fmaf(v[b].y, h, o.y), fmaf(v[b].z, h, o.z), fmaf(v[b].w, h, o.w));
      }
    };
    float2 st[kBatch];
    float4 v[kBatch];
    for (int i = g0 + sub; i <= j.z; i += kBatch * step) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = i + b * step;
        const int64_t part = ((int64_t)(k * a.gang + member) * 2 + (k == g0 ? 1 : 0)) * a.part_rows + row;
        st[b] = make_float2(kRefStart, 0.f);
        v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= j.z) {
          st[b] = stats[part];
          v[b] = *reinterpret_cast<const float4*>(a.parts + part * DP + 4 * lane);
        }
      }
      add(st, v);
    }
    if (together) {                          // one item a CTA
      s_o[group][lane] = o;
      if (lane == 0) s_stat[group] = make_float2(top, l);
      __syncthreads();
      if (group > 0) return;
      top = kRefStart;
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kGroups; g += kBatch) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) st[b] = s_stat[g + b], v[b] = s_o[g + b][lane];
        add(st, v);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = (row0 + row) / a.group, g = row0 + row - tok * a.group;
    if (4 * lane < a.head_dim)
      *reinterpret_cast<uint2*>(
          a.out + ((int64_t)(first + tok) * a.q_heads + head * a.group + g) * a.head_dim + 4 * lane) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  }
}

// How a call's work is laid out.
struct Plan {
  int dp, rows, passes, gang, gangs, part_rows, q_rows, q_bufs, q_box, slots, warps;
  int64_t joins_bytes() const { return ((int64_t)gangs * gang * 16 + 127) / 128 * 128; }
  int64_t bytes() const { return joins_bytes() + (int64_t)gangs * gang * 2 * part_rows * (dp + 2) * 4; }
};
Plan plan_of(int32_t max_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  Plan p;
  const int group = num_q_heads / num_kv_heads, rows = max_rows * group;
  p.dp = head_dim <= 64 ? 64 : 128;
  p.rows = rows > kTile ? 2 : 1;
  p.passes = (rows + p.rows * kTile - 1) / (p.rows * kTile);
  const int segs = num_kv_heads * p.passes;
  // the largest divisor of the (KV head, pass) pairs up to 8 (measured above)
  p.gang = segs < 8 ? segs : 8;
  while (segs % p.gang != 0) --p.gang;
  const int ctas = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  p.gangs = ctas / p.gang;
  if (p.gangs < 1) p.gang = p.gangs = 1;
  p.part_rows = rows < p.rows * kTile ? rows : p.rows * kTile;
  const int tile_rows = rows < kTile ? rows : kTile;
  p.q_rows = (tile_rows + 7) / 8 * 8;
  p.q_box = tile_rows % group == 0 ? tile_rows / group : 0;
  p.warps = (tile_rows + 31) / 32;
  const int head = kHead;
  const int q_bytes = (p.q_rows * p.dp * 2 * p.rows + 1023) / 1024 * 1024, slot = kTile * p.dp * 2;
  const int want = p.dp == 64 ? 10 : 5;
  p.q_bufs = head + 2 * q_bytes + want * slot <= kSmemMax ? 2 : 1;
  p.slots = (kSmemMax - head - p.q_bufs * q_bytes) / slot;
  if (p.slots > 12) p.slots = 12;
  return p;
}

template <int DP, int kRows, bool kTma>
int launch(const TreeArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
           cudaStream_t stream) {
  auto kernel = attention_tree_kernel<DP, kRows, kTma>;
  const int q_bytes = (a.q_bufs * kRows * a.q_rows * DP * 2 + 1023) / 1024 * 1024;
  // Q's matrix instructions read whole tiles of 128 rows: the ring lies behind it
  const int smem = kHead + q_bytes + a.slots * Layout<DP>::kSlot;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return KV_ECUDA;
  const unsigned ctas = (unsigned)(a.gangs * a.gang);
  const int rc = launch_pdl(kernel, ctas, kThreadsOf<kRows>, smem, stream, a, q_map, k_map, v_map);
  if (rc != KV_OK) return rc;
  return launch_pdl(join_tree_kernel<DP, kRows>, kJoins * ctas, kJoinThreads, 0, stream, a);
}

template <int DP, int kRows>
int launch(const TreeArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
           cudaStream_t stream) {
  return a.box > 1 ? launch<DP, kRows, true>(a, q_map, k_map, v_map, stream)
                   : launch<DP, kRows, false>(a, q_map, k_map, v_map, stream);
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
  return rc != KV_OK ? rc : plan_of(max_rows, num_q_heads, num_kv_heads, head_dim).bytes();
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
  if (num_blocks > INT32_MAX / block_size || (int64_t)num_kv_heads * head_dim > INT32_MAX / 2)
    return KV_EUNSUPPORTED;  // tokens of the pool and bytes of a row are counted in 32 bits
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
  // the largest box of 8, 16, .. tokens that never crosses a block
  int box = 1;
  if (block_size % 8 == 0)
    for (box = 8; box < kTile && block_size % (2 * box) == 0;) box *= 2;
  const Plan p = plan_of(max_rows, num_q_heads, num_kv_heads, head_dim);
  CUtensorMap q_map = {}, k_map = {}, v_map = {};
  const int64_t tokens = num_blocks * block_size, kv_row = (int64_t)num_kv_heads * head_dim;
  const int group = num_q_heads / num_kv_heads;
  if (box > 1 && (!rows_map(&k_map, k_layer, kv_row, tokens, num_kv_heads, head_dim, 1, box) ||
                  !rows_map(&v_map, v_layer, kv_row, tokens, num_kv_heads, head_dim, 1, box)))
    return KV_ECUDA;
  const bool q_boxes = box > 1 && p.q_box > 0 && query_stride < ((int64_t)1 << 39);  // bytes below 2^40
  if (q_boxes && !rows_map(&q_map, query, query_stride, num_rows, num_q_heads, head_dim, group, p.q_box))
    return KV_ECUDA;
  const TreeArgs a{static_cast<const __nv_bfloat16*>(query), query_stride,
                   reinterpret_cast<const __nv_bfloat16*>(k_layer),
                   reinterpret_cast<const __nv_bfloat16*>(v_layer), num_blocks,
                   BlockDiv::make(block_size), num_q_heads, num_kv_heads, head_dim,
                   group, block_table, table_stride, q_start_loc, span_start,
                   context_len, tree_mask, num_reqs, num_rows, max_rows,
                   fminf(scale * 1.44269504088896340736f, FLT_MAX),
                   static_cast<__nv_bfloat16*>(out), d_err, p.passes, p.gang, p.gangs, p.part_rows,
                   p.q_rows, p.q_bufs, q_boxes ? p.q_box : 0, p.slots, box, p.warps, static_cast<int4*>(workspace),
                   reinterpret_cast<float*>(static_cast<char*>(workspace) + p.joins_bytes())};
  if (p.dp == 64)
    return p.rows == 1 ? launch<64, 1>(a, q_map, k_map, v_map, stream) : launch<64, 2>(a, q_map, k_map, v_map, stream);
  return p.rows == 1 ? launch<128, 1>(a, q_map, k_map, v_map, stream) : launch<128, 2>(a, q_map, k_map, v_map, stream);
}
