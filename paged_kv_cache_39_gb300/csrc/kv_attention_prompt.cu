// kv_attention_prompt.cu -- causal attention of packed sequences with grouped
// heads, on the matrix unit.
//
// Mathematics.  Request r holds query rows i < m and key rows j < n; row i sees
// the keys j < seen_i = i + n - m + 1:
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c q_i . k_j - ref_i),
// c = scale * log2(e).  One pass over the keys with a running reference ref_i:
// it is the row's maximum when it was last raised, and is raised (with the
// accumulator rescaled) only when a new maximum passes it by more than 8, so
// that p stays below 2^8 and the rescale almost never runs.  Logits, weights,
// sums and outputs are held in 32 bits; p is rounded to bf16 for its product
// with V (the matrix unit takes both operands in one type), at most 2^-8 of a
// weight; the sum takes p before that rounding.
//
// GPU shape.  A CTA owns 2 tiles of 128 query rows and one KV head.  A tile's rows
// are tq = 128 / group tokens x the group's heads, so every head of the group
// shares the K and V tiles and rows of one tile end at almost the same key
// whatever the group is.  Roles by warp:
//   0-3, 4-7  softmax of tile 0 / 1: one row per thread, so no shuffles; also the
//             rescale and the epilogue of its tile
//   8         TMA: Q, then K and V tiles of 128 keys into a ring; finds the next pair
//   9         issues the matrix instructions: S = Q K^T (both operands in shared
//             memory), O += P V (P from tensor memory, over the S it came from)
//   10, 11    check V tiles at the causal edge (below)
// While one tile's softmax runs, the matrix unit works for the other.  Tensor
// memory: S0 S1 (128 columns each, P in place), O0 O1: all 512 columns, hence one
// CTA per SM.
//
// Hidden keys.  A hidden logit is replaced, so a NaN there is gone, but 0 * NaN in
// P V is NaN.  So in the tiles where some key is hidden from some row (one to three
// per pair), V values that are not finite are set to 0 in shared memory, and the
// first key that held one is kept per channel: rows that see that key
// get NaN in the epilogue.  Rows behind the sequence are set to 0 outright.
//
// Few rows behind many keys.  Where the tile pairs leave SMs idle, a cluster of up to 16 CTAs
// takes a pair, each CTA a run of its key tiles.  The CTAs then leave their accumulators, references
// and sums in their own shared memory, and each joins a share of the rows from all of them:
//   o_i = sum_c f_c O_c / sum_c f_c s_c,  f_c = 2^(ref_c - max ref).
// No workspace, no atomics: the same call gives the same bits.  The join costs 3 us; 16 tokens
// behind 8192 take 15 us instead of 74, behind 65536 56 instead of 558.
//
// Many pairs.  A CTA that runs takes over the pairs of CTAs that wait (see kv_tc.cuh), so that
// the start of the next pair (search, loads, first scores) overlaps the end of this one: 64 prompts
// of 128 tokens 74 -> 40 us, 256 of 64 207 -> 72.
//
// Measured (32 query heads, 8 KV heads of 128 channels): one prompt of 32768 tokens 5.3 to 5.4 ms
// (1630 to 1660 TFLOP/s, near the card's power limit, 1.92 GHz), 16 chunks of 9 to 1855 tokens behind
// up to 7685 366 us (1370 TFLOP/s), 77 tokens 7.7 us.  Per 128 keys a CTA's two tiles take 2900
// cycles: 2048 of matrix instructions; a tile's softmax is 1140, beside the other tile's products,
// and its S, softmax and O follow one another with the barriers' times between them.  The mixed
// chunks' 32840 such steps are 311 us of it at 2.07 GHz (335 at 1.92), in this order on 152 SMs; the
// rest is 4 to 8 us for each of a CTA's seven pairs: edge tiles, hand-over, output.
#include <cuda_bf16.h>

#include <cfloat>
#include <mutex>
#include <type_traits>

#include "kv_tc.cuh"

namespace kvp {
namespace {

constexpr int kTile = 128;                 // query rows of a tile, keys of a K/V tile
constexpr int kThreads = 384;
constexpr int kScrubThreads = 64;
constexpr int kReaders = 11;               // warps that a work description is passed on to
constexpr int kEdges = 3;                  // K/V tiles a CTA's rows see in part: 256 tokens span at most 3
constexpr int kMaxKeys = 1 << 24;         // of a request: the longest wait in a CTA is the edge's, for all
                                          // tiles before it, 0.2 s at this length; waits end at 1 s
constexpr int kL2Share = 48 << 20;        // K and V of all heads stay in the L2 up to this (of 129 MB)
constexpr int kSplitMax = 16;              // the largest cluster
constexpr int kSplitFrom = 6;              // K/V tiles from which on a split pays for its join (3 us)
constexpr int kSplitTiles = 2;             // least of them that a CTA takes
constexpr float kLazy = 8.0f;              // log2 of the most a weight may pass the reference
constexpr float kRefStart = -1e30f;        // of a row with no finite logit yet: below every other
// Registers: 384 threads x 168 at launch = 256 x 200 + 128 x 104.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;

struct PromptArgs {
  const int32_t* q_start;
  const int32_t* k_start;
  int32_t num_reqs, nq, nk, q_heads, kv_heads, head_dim;
  int32_t group, tq;       // query heads per KV head, tokens per tile
  int32_t items;           // upper bound of (request, tile pair), the grid's extent per head
  int32_t split;           // CTAs of a cluster, which share a tile pair's keys
  int32_t by_head;         // all pairs of one head come before the next head's
  float scale_log2;
  __nv_bfloat16* out;
  int32_t* err;
  // the self-test's: which role waits for nothing, at which of its CTA's items, for how long
  int32_t stall_role, stall_item;
  int64_t stall_ns;
};
enum Role { kLoader, kIssuer, kValueCheck, kSoftmax };  // kSoftmax + tile

// One step of a transposition over lanes: with the lane `mask` away, a for its b (the lower of the
// two lanes keeps its a, the higher its b).
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b, bool high, int mask) {
  const uint32_t got = __shfl_xor_sync(kFull, high ? a : b, mask);
  a = high ? got : a;
  b = high ? b : got;
}
__device__ __forceinline__ void exchange(uint4& a, uint4& b, bool high, int mask) {
  exchange(a.x, b.x, high, mask);
  exchange(a.y, b.y, high, mask);
  exchange(a.z, b.z, high, mask);
  exchange(a.w, b.w, high, mask);
}

template <int DP>
struct Smem {
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBars = kRing + kSlots * kTileBytes;
  // full[slots], empty[slots], edge[2][3], v_ok[2][3], q_full, q_free, s_full[2], p_full[2][2],
  // o_full[2], scrubbed, written[2], ready, drain, stolen, work_full[2], work_free[2]
  static constexpr int kNumBars = 2 * kSlots + 4 * kEdges + 20;
  static constexpr int kBad = kBars + kNumBars * 8;         // int[DP]: first key not finite
  static constexpr int kMisc = kBad + DP * 4;
  static constexpr int kAnswer = kMisc + 16;                // 16 bytes: the work taken over
  static constexpr int kWork = kAnswer + 16;                // Work[2]
  static constexpr int kOrder = kWork + 64;                 // uint16_t[kThreads]: requests by keys
  static constexpr int kBytes = kOrder + kThreads * 2 + 1024;  // + alignment of the base
  static_assert(kBars % 16 == 0 && kNumBars % 2 == 0 && kSlots <= 8, "");
  // for the join of a split: fp32 accumulators and (reference, sum) of 2 x 128 rows, where Q, K
  // and V were
  static constexpr int kStats = 2 * kTile * DP * 4;
  static_assert(kStats + 2 * kTile * 8 <= kBars, "");
};

struct Work {
  int32_t q0, k0, m, n;  // the request's first rows and lengths; m = 0: no work
  int32_t t0;            // first token of the pair of tiles
  int32_t head;
};

// What of it a CTA does.
struct Item : Work {
  int32_t ahead;       // keys before the first query's own
  int32_t last;        // last token
  int32_t tiles;       // K/V tiles that the last token sees
  int32_t whole;       // of them, those that every row sees whole
  int32_t parts;       // CTAs that share them
  int32_t first, end;  // this CTA's
  bool two;            // both tiles of the pair have tokens
  __device__ __forceinline__ Item(const Work& w, const PromptArgs& a, int split, int rank) : Work(w) {
    ahead = n - m;
    last = min(t0 + 2 * a.tq, m) - 1;
    const int keys = max(0, min(n, ahead + last + 1));
    tiles = (keys + kTile - 1) / kTile;
    whole = max(0, ahead + t0 + 1) / kTile;
    parts = split > 1 && tiles >= kSplitFrom ? min(split, tiles / kSplitTiles) : 1;
    first = rank < parts ? tiles * rank / parts : 0;
    end = rank < parts ? tiles * (rank + 1) / parts : 0;
    two = t0 + a.tq < m;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Behind a role's last wait, read and issue: all roles of the CTA have come so far.
__device__ __forceinline__ void roles_met() {
  tc_fence_before();
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  tc_fence_after();
}

// Three kernels of one body, so that none has another's registers and code in its way (with the
// join in all: 5.63 instead of 5.46 ms at 32768 tokens).
enum Mode {
  kOneWave,    // every CTA has one item
  kManyWaves,  // those that run take over the work of those that wait
  kClusters,   // `split` CTAs share an item
};
template <int DP, Mode kMode, bool kStall>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map, PromptArgs a) {
  using L = Smem<DP>;
  constexpr bool kSplit = kMode == kClusters, kSteal = kMode == kManyWaves;
  extern __shared__ unsigned char raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* full = bars;
  uint64_t* empty = full + L::kSlots;
  uint64_t* edge = empty + L::kSlots;  // [item & 1][tile - whole]
  uint64_t* v_ok = edge + 2 * kEdges;
  uint64_t* q_full = v_ok + 2 * kEdges;
  uint64_t* q_free = q_full + 1;
  uint64_t* s_full = q_free + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 4;
  uint64_t* scrubbed = o_full + 2;
  uint64_t* written = scrubbed + 1;
  uint64_t* ready = written + 2;
  uint64_t* drain = ready + 1;
  uint64_t* stolen = drain + 1;
  uint64_t* work_full = stolen + 1;  // [item & 1]
  uint64_t* work_free = work_full + 2;
  int* bad = reinterpret_cast<int*>(smem + L::kBad);
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  volatile int* any_bad = misc + 2;
  Work* s_work = reinterpret_cast<Work*>(smem + L::kWork);
  uint16_t* order = reinterpret_cast<uint16_t*>(smem + L::kOrder);
  __shared__ uint64_t nothing;  // kStall: a barrier that nobody arrives on
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform for the compiler, too
  if constexpr (kStall) {
    if (tid == 0) mbar_init(&nothing, 1);
  }

  if (tid < L::kNumBars) {
    const uint64_t* b = &bars[tid];
    int count = 1;
    if (b >= v_ok && b < v_ok + 2 * kEdges) count = kScrubThreads;
    if (b == scrubbed || b == ready) count = kScrubThreads;
    if (b >= p_full && b < p_full + 4) count = kTile / 32;  // one arrival a warp
    if (b >= written && b < written + 2) count = kTile / 32;
    if (b >= work_free && b < work_free + 2) count = kReaders;
    mbar_init(&bars[tid], count);
    mbar_fence_init();
  }
  if (tid == 0) {
    *abort = 0;
    *any_bad = 0;
    s_work[0] = Work{0, 0, 0, 0, 0, 0};  // of a CTA that no pair is left for
  }
  if (tid < DP) bad[tid] = INT32_MAX;
  pdl_allow_next();
  pdl_wait();
  if (warp == 9) tmem_alloc(tmem_ptr, 512);  // not before: what runs ahead may need it to end

  // Which pair of tiles is this?  The pairs are numbered by request, those with the most keys
  // first (as long as a thread can rank each of them), and inside a request from its last
  // tokens, which see the most keys, to its first: CTAs start in this order, so the long ones do
  // not end up alone at the end (16 chunks of 9 to 1855 tokens: 468 -> 434 us).  The heads of a
  // pair are neighbours, so the request's K and V are in L2 for all of them.  Every thread
  // counts the pairs of its share of the requests, a block-wide scan places them, the thread
  // that owns pair `want` describes it.
  const bool rank = a.num_reqs > 1 && a.num_reqs <= kThreads;
  const int pair_tokens = 2 * a.tq;
  const int split = kSplit ? a.split : 1;
  const int rank_in = kSplit ? (int)(blockIdx.x % (unsigned)split) : 0;
  auto head_of = [&](int block) { return a.by_head ? block / a.items : block % a.kv_heads; };
  auto want_of = [&](int block) { return a.by_head ? block % a.items : block / a.kv_heads; };
  auto pairs = [&](const Work& x) { return (int)(((int64_t)x.m + pair_tokens - 1) / pair_tokens); };
  uint32_t err = 0;
  auto describe = [&](int r) {  // request r, or one without rows where it is not valid
    const int q0 = a.q_start[r], q1 = a.q_start[r + 1], k0 = a.k_start[r], k1 = a.k_start[r + 1];
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.nq && k0 >= 0 && k1 >= k0 && k1 <= a.nk &&
                    k1 - k0 <= kMaxKeys;
    if (!ok) err |= KV_ERR_BAD_QSL;
    return ok ? Work{q0, k0, q1 - q0, k1 - k0, 0, 0} : Work{0, 0, 0, 0, 0, 0};
  };
  {
    __shared__ int64_t warp_sum[kThreads / 32];
    const int block = (int)(blockIdx.x / (unsigned)split), want = want_of(block);
    int* keys_of = reinterpret_cast<int*>(smem);                     // [num_reqs], and
    int4* ranked = reinterpret_cast<int4*>(smem + kThreads * sizeof(int));  // the same: where Q will be
    const int per = (a.num_reqs + kThreads - 1) / kThreads;
    const int r_lo = min(a.num_reqs, tid * per), r_hi = min(a.num_reqs, r_lo + per);
    Work mine = {0, 0, 0, 0, 0, 0};  // with `rank`: the request of this thread's rank
    int64_t count = 0;  // 64 bits: requests that claim the same rows may count more than there are
    if (rank) {
      if (tid < a.num_reqs) {
        mine = describe(tid);
        keys_of[tid] = mine.n;
      }
      __syncthreads();
      if (tid < a.num_reqs) {
        int before = 0;
        for (int r = 0; r < a.num_reqs; ++r)
          before += keys_of[r] > mine.n || (keys_of[r] == mine.n && r < tid);
        ranked[before] = make_int4(mine.q0, mine.k0, mine.m, mine.n);
        order[before] = (uint16_t)tid;
      }
      __syncthreads();
      if (tid < a.num_reqs) {
        const int4 x = ranked[tid];
        mine = Work{x.x, x.y, x.z, x.w, 0, 0};
        count = pairs(mine);
      }
      fence_proxy_async_smem();  // before TMA writes Q there
    } else {
      for (int r = r_lo; r < r_hi; ++r) count += pairs(describe(r));
    }
    const int64_t incl = warp_inclusive_scan<int64_t>(count);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t at = incl - count;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    if (want >= at && want < at + count) {
      if (!rank) {
        int r = r_lo;
        for (mine = describe(r); want >= at + pairs(mine); mine = describe(++r)) at += pairs(mine);
      }
      mine.t0 = (pairs(mine) - 1 - (int)(want - at)) * pair_tokens;
      mine.head = head_of(block);
      s_work[0] = mine;
    }
    if (blockIdx.x == 0) report(a.err, err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_ptr, 0);

  // A CTA goes on with the work of CTAs that have not started: the loading warp takes it over
  // (the hardware hands a CTA that waits to another one only once, in launch order) while the
  // others still compute, and passes it on in s_work[item & 1].  All barriers' phases run on from
  // item to item, so the next item's Q, K and V are loaded and its first scores computed while this
  // one's last weights and outputs are.
  auto read = [&](int item) {  // the same in every lane: tell the compiler
    const Work* p = &s_work[item & 1];
    Work w;
    w.q0 = __shfl_sync(kFull, p->q0, 0);
    w.k0 = __shfl_sync(kFull, p->k0, 0);
    w.m = __shfl_sync(kFull, p->m, 0);
    w.n = __shfl_sync(kFull, p->n, 0);
    w.t0 = __shfl_sync(kFull, p->t0, 0);
    w.head = __shfl_sync(kFull, p->head, 0);
    return w;
  };
  // Readers: the item after `item`, m = 0 behind the last one (or when a wait ran out).
  auto following = [&](int item) {
    Work none = {0, 0, 0, 0, 0, 0};
    if (!kSteal) return none;
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_free[item & 1]);
    const bool ok = mbar_wait_role(&work_full[(item + 1) & 1], (item >> 1) & 1, abort);
    return __all_sync(kFull, ok) ? read(item + 1) : none;
  };

  // The self-test: this role gives up at this item.
  auto stalled = [&](int role, int item) {
    if constexpr (kStall) {
      if (role == a.stall_role && item == a.stall_item)
        return !mbar_wait_role(&nothing, 0, abort, (uint64_t)a.stall_ns);
    }
    return false;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // -------------------------------------------------------------- TMA
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
      }
      int slot = 0, turn = 0, items = 0, loaded = 0;
      uint32_t edge_at = 0, edge_used = 0;  // bits: parities of the next use; used at all
      int base = 0;             // where the search for the next item goes on: requests and
      int64_t base_at = 0;      // pairs before it
      bool ok = true, asked = false;
      Work w = read(0);
      for (int item = 0; w.m > 0; ++item) {
        if (stalled(kLoader, item)) break;
        const Item x(w, a, split, rank_in);
        if (x.end > x.first) {
          if (loaded > 0) ok = __all_sync(kFull, mbar_wait_role(q_free, (loaded - 1) & 1, abort));
          if (!ok) break;
          if (leader) {
            const uint32_t q_bytes = (uint32_t)(a.group * a.tq) * 128u * (DP / 64);
            mbar_arrive_expect_tx(q_full, x.two ? 2 * q_bytes : q_bytes);
            for (int t = 0; t < (x.two ? 2 : 1); ++t)
              for (int c = 0; c < DP / 64; ++c)
                tma_load_3d(smem + L::kQ + t * L::kTileBytes + c * (kTile * 128), &q_map, 64 * c,
                            x.head * a.group, x.q0 + x.t0 + t * a.tq, q_full);
          }
          ++loaded;
#pragma unroll 1
          for (int u = 2 * x.first; u < 2 * x.end; ++u) {  // K and V tiles alternate in the ring
            if (turn > 0) {
              ok = __all_sync(kFull, mbar_wait_role(&empty[slot], (turn - 1) & 1, abort));
              if (!ok) break;
            }
            const bool is_v = u & 1;
            const int j = u >> 1;
            const int e = is_v && j >= x.whole ? (item & 1) * kEdges + j - x.whole : -1;
            uint64_t* bar = e >= 0 ? &edge[e] : &full[slot];
            if (leader) {
              if (e >= 0) mbar_arrive(&full[slot]);  // its phases count the turns of the ring
              mbar_arrive_expect_tx(bar, L::kTileBytes);
              for (int c = 0; c < DP / 64; ++c)
                tma_load_3d(smem + L::kRing + slot * L::kTileBytes + c * (kTile * 128),
                            is_v ? &v_map : &k_map, 64 * c, x.head, x.k0 + j * kTile, bar);
            }
            if (e >= 0) {
              edge_at ^= 1u << e;
              edge_used |= 1u << e;
            }
            if (++slot == L::kSlots) {
              slot = 0;
              ++turn;
            }
          }
          if (!ok) break;
        }
        if (!kSteal) break;
        // the next item: that of a CTA that waits, if any does
        w.m = 0;
        for (bool more = true; more && w.m == 0;) {
          if (leader) {
            fence_proxy_async_smem();  // the last answer was read
            mbar_arrive_expect_tx(stolen, 16);
            take_over(smem + L::kAnswer, stolen);
          }
          asked = true;
          ok = mbar_wait_role(stolen, items & 1, abort);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          asked = false;
          ++items;
          int block;
          more = __all_sync(kFull, taken_over(smem + L::kAnswer, &block));
          block = __shfl_sync(kFull, block, 0);
          if (!more) break;
          const int want = want_of(block);
          if (want < base_at) base = 0, base_at = 0;
          for (; base < a.num_reqs; base += 32) {  // 32 requests at a time
            Work mine = {0, 0, 0, 0, 0, 0};
            if (base + lane < a.num_reqs) mine = describe(rank ? order[base + lane] : base + lane);
            const int count = pairs(mine);
            const int64_t incl = warp_inclusive_scan<int64_t>(count);
            const int64_t at = base_at + incl - count;
            const uint32_t found = __ballot_sync(kFull, want >= at && want < at + count);
            if (found != 0) {
              const int src = __ffs(found) - 1;
              mine.t0 = (count - 1 - (int)(want - at)) * pair_tokens;
              w.q0 = __shfl_sync(kFull, mine.q0, src);
              w.k0 = __shfl_sync(kFull, mine.k0, src);
              w.m = __shfl_sync(kFull, mine.m, src);
              w.n = __shfl_sync(kFull, mine.n, src);
              w.t0 = __shfl_sync(kFull, mine.t0, src);
              w.head = head_of(block);
              break;
            }
            base_at += __shfl_sync(kFull, incl, 31);
          }
        }
        // s_work[..] is free once all have finished the item before this one
        if (ok && item > 0) {
          ok = mbar_wait_role(&work_free[(item - 1) & 1], ((item - 1) >> 1) & 1, abort);
          ok = __all_sync(kFull, ok);
        }
        if (!ok) break;
        if (leader) {
          s_work[(item + 1) & 1] = w;
          mbar_arrive(&work_full[(item + 1) & 1]);
        }
        __syncwarp();
      }
      // Where a wait ran out, wait (with a bound) for the copies still in flight: only now, when
      // the other roles have left, is it known that none did, and no shared memory is given up or
      // written by a split's join before this.
      roles_met();
      if (__any_sync(kFull, *abort != 0)) {
        if (loaded > 0) mbar_wait_bounded(q_full, (loaded - 1) & 1);
        if (asked) mbar_wait_bounded(stolen, items & 1);
        for (int i = 0; i < L::kSlots; ++i) {
          const int uses = turn + (i < slot ? 1 : 0);
          if (uses > 0) mbar_wait_bounded(&full[i], (uses - 1) & 1);
        }
        for (int e = 0; e < 2 * kEdges; ++e)
          if ((edge_used >> e) & 1u) mbar_wait_bounded(&edge[e], ((edge_at >> e) & 1u) ^ 1u);
      }
    } else if (warp == 9) {
      // -------------------------------------------------------------- matrix instructions
      constexpr uint32_t s_desc = mma_desc(128, kTile, false), o_desc = mma_desc(128, DP, true);
      constexpr uint32_t kSlotStep = L::kTileBytes >> 4;  // descriptors count 16 bytes
      const uint64_t q_at = smem_desc(smem_addr(smem + L::kQ), 16);
      const uint64_t k_at = smem_desc(smem_addr(smem + L::kRing), 16);
      const uint64_t v_at = smem_desc(smem_addr(smem + L::kRing), kTile * 128);
      const bool leader = elect_one();
      auto scores = [&](int t, int slot) {
        const uint64_t qd = q_at + t * kSlotStep, kd = k_at + slot * kSlotStep;
        const uint32_t d = tmem + t * kTile;
        if (leader) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint32_t off = ((k / 4) * (kTile * 128) + (k % 4) * 32) >> 4;
            mma_ss(d, qd + off, kd + off, s_desc, k > 0);
          }
          mma_commit(&s_full[t]);
        }
      };
      auto values = [&](int t, int slot, bool add, int half) {
        const uint64_t vd = v_at + slot * kSlotStep + half * ((kTile / 2 * 128) >> 4);
        const uint32_t d = tmem + 2 * kTile + t * DP, p = tmem + t * kTile + half * (kTile / 4);
        if (leader) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_ts(d, p + k * 8, vd + k * (2048 >> 4), o_desc, add || k > 0);
        }
      };
      int sv = 0, sk = 0, pv = 0, pk = 0;  // slots of V and the next K, parities of their phases
      int loaded = 0;
      uint32_t p_at = 0, v_ok_at = 0;      // bits: parities of the next waits (p_full: per tile)
      bool ok = true;
      Work w = read(0);
      for (int item = 0; w.m > 0; ++item) {
        if (stalled(kIssuer, item)) break;
        const Item x(w, a, split, rank_in);
        if (x.end > x.first) {
          ok = mbar_wait_role(q_full, loaded & 1, abort) && mbar_wait_role(&full[sk], pk, abort);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          ++loaded;
          tc_fence_after();
          scores(0, sk);
          if (x.two) scores(1, sk);
          if (leader) {
            mma_commit(&empty[sk]);
            if (x.end - x.first == 1) mma_commit(q_free);
          }
          const int nt = x.two ? 2 : 1;
          auto step = [](int& slot, int& phase) {
            if (++slot == L::kSlots) {
              slot = 0;
              phase ^= 1;
            }
          };
          sv = sk, pv = pk;
          step(sv, pv);
          sk = sv, pk = pv;
          step(sk, pk);
          auto advance = [&]() {
            sv += 2;
            sk += 2;
            if (sv >= L::kSlots) {
              sv -= L::kSlots;
              pv ^= 1;
            }
            if (sk >= L::kSlots) {
              sk -= L::kSlots;
              pk ^= 1;
            }
          };
          auto tile = [&](int t, uint32_t phase, bool add, bool more) {
            if (!mbar_wait_role(&p_full[2 * t], phase, abort)) return false;
            tc_fence_after();
            values(t, sv, add, 0);
            if (!mbar_wait_role(&p_full[2 * t + 1], phase, abort)) return false;
            tc_fence_after();
            values(t, sv, true, 1);
            if (more) scores(t, sk);  // in issue order behind the P V that reads what it overwrites
            else if (leader) mma_commit(&o_full[t]);
            return true;
          };
          int j = x.first;
          bool add = false;
          // the usual step by itself, with as little as can be between the waits: what the issue
          // takes longer, the matrix unit waits (5.9 ms at 32768 tokens with the loop below alone)
          if (x.two) {
#pragma unroll 1
            for (; j + 2 < x.end && j < x.whole; ++j) {
              ok = mbar_wait_role(&full[sv], pv, abort) && mbar_wait_role(&full[sk], pk, abort) &&
                   tile(0, p_at & 1, add, true) && tile(1, p_at >> 1, add, true);
              ok = __all_sync(kFull, ok);  // also keeps the lanes within one step of each other
              if (!ok) break;
              if (leader) {
                mma_commit(&empty[sv]);
                mma_commit(&empty[sk]);
              }
              p_at ^= 3;
              add = true;
              advance();
            }
          }
#pragma unroll 1
          for (; ok && j < x.end; ++j) {
            const bool more = j + 1 < x.end;
            // at the causal edge V is waited for through the warps that check it
            if (j < x.whole) {
              ok = mbar_wait_role(&full[sv], pv, abort);
            } else {
              const int e = (item & 1) * kEdges + j - x.whole;
              ok = mbar_wait_role(&v_ok[e], (v_ok_at >> e) & 1, abort);
              v_ok_at ^= 1u << e;
            }
            if (ok && more) ok = mbar_wait_role(&full[sk], pk, abort);
#pragma unroll 1
            for (int t = 0; ok && t < nt; ++t) ok = tile(t, (p_at >> t) & 1, add, more);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            if (leader) {
              mma_commit(&empty[sv]);
              if (more) mma_commit(&empty[sk]);
              if (more && j + 2 == x.end) mma_commit(q_free);
            }
            p_at ^= x.two ? 3 : 1;
            add = true;
            if (more) advance();  // else sk is the next item's first K
          }
          if (!ok) break;
        }
        w = following(item);
      }
      // The matrix unit arrives on barriers on its own time: none of its arrivals (the last slots',
      // which nobody waits for) may come after the CTA's shared memory has gone to another.  It
      // takes them in order, so the last one stands for all.
      __syncwarp();
      if (leader) mma_commit(drain);
      mbar_wait_bounded(drain, 0);
      roles_met();
    } else {
      // -------------------------------------------------------------- V at the causal edge
      const int st = tid - 10 * 32;
      int slot = 0, done = 0;
      uint32_t edge_at = 0, written_at = 0;
      bool both = false;  // the item before had two tiles
      Work w = read(0);
      for (int item = 0; w.m > 0; ++item) {
        if (stalled(kValueCheck, item)) break;
        const Item x(w, a, split, rank_in);
        if (x.end > x.first) {
          bool ok = true;
          if (done > 0) {  // the item before is written: its `bad` goes
            ok = mbar_wait_role(&written[0], written_at & 1, abort);
            if (ok && both) ok = mbar_wait_role(&written[1], written_at >> 1, abort);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            written_at ^= both ? 3 : 1;
            for (int i = st; i < DP; i += kScrubThreads) bad[i] = INT32_MAX;
            if (st == 0) *any_bad = 0;
            mbar_arrive(ready);
            ok = __all_sync(kFull, mbar_wait_role(ready, (done - 1) & 1, abort));
            if (!ok) break;
          }
          ++done;
          both = x.two;
          for (int j = max(x.first, x.whole); j < x.end; ++j) {
            const int e = (item & 1) * kEdges + j - x.whole;
            ok = mbar_wait_role(&edge[e], (edge_at >> e) & 1, abort);
            edge_at ^= 1u << e;
            if (!ok) break;
            unsigned char* tile =
                smem + L::kRing + ((slot + 2 * (j - x.first) + 1) % L::kSlots) * L::kTileBytes;
#pragma unroll 1
            for (int r = st; r < kTile; r += kScrubThreads) {
              const int key = j * kTile + r;
              // the row's 16-byte pieces, the row's own one first: no two of 8 rows share a bank
              auto piece = [&](int i) {
                return reinterpret_cast<uint4*>(tile + (i / 8) * (kTile * 128) + r * 128 + ((i + r) & 7) * 16);
              };
              if (key >= x.n) {
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) *piece(i) = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint32_t most = 0;  // the largest magnitudes, two to a word; 0x7f80 and up: not finite
#pragma unroll
              for (int i = 0; i < DP / 8; ++i) {
                const uint4 y = *piece(i);
                most = __vmaxu2(most, __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                               __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
              }
              if ((most & 0xffffu) < 0x7f80u && most < 0x7f800000u) continue;
#pragma unroll 1
              for (int i = 0; i < DP / 8; ++i) {
                uint4 y = *piece(i);
                uint32_t* q = reinterpret_cast<uint32_t*>(&y);
                const int channel = (i / 8) * 64 + (((i + r) & 7) ^ (r & 7)) * 8;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  if ((q[c] & 0x7f80u) == 0x7f80u) {
                    atomicMin(&bad[channel + 2 * c], key);
                    q[c] &= 0xffff0000u;
                  }
                  if ((q[c] & 0x7f800000u) == 0x7f800000u) {
                    atomicMin(&bad[channel + 2 * c + 1], key);
                    q[c] &= 0xffffu;
                  }
                }
                *piece(i) = y;
              }
              *any_bad = 1;
            }
            fence_proxy_async_smem();
            mbar_arrive(&v_ok[e]);
          }
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          mbar_arrive(scrubbed);
          slot = (slot + 2 * (x.end - x.first)) % L::kSlots;
        }
        w = following(item);
      }
      roles_met();
    }
    if constexpr (kSplit) {  // the softmax warps' join
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;  // the tile
    const int row = tid & 127;
    const int tok = row / a.group, g = row - tok * a.group;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes, in bits 16..
    const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 2 * kTile + t * DP;
    const float c = a.scale_log2;
    uint32_t s_phase = 0, o_phase = 0;
    int done = 0;
    Work w = read(0);
    for (int item = 0; w.m > 0; ++item) {
      if (stalled(kSoftmax + t, item)) break;
      const Item x(w, a, split, rank_in);
      const bool work = x.end > x.first;
      if (x.tiles == 0 && rank_in == 0) {  // no query here sees a key
        const int64_t dense = (int64_t)a.group * a.head_dim;
        const int vecs = (int)(dense / 8);
        for (int64_t i = tid; i < (int64_t)(x.last + 1 - x.t0) * vecs; i += 256) {
          const int64_t at = x.q0 + x.t0 + i / vecs;
          reinterpret_cast<uint4*>(a.out + at * a.q_heads * a.head_dim + x.head * dense)[i % vecs] =
              make_uint4(0, 0, 0, 0);
        }
      }
      if (work && (t == 0 || x.two)) {
        // ------------------------------------------------------------ softmax
        const int i = x.t0 + t * a.tq + tok;  // token in the request
        const bool mine = tok < a.tq && i < x.m;
        const int seen = min(x.n, x.ahead + i + 1);
        s_phase -= x.first;
        float ref = 0.f;
        uint64_t part[2] = {0, 0};  // sums of weights, two by two
        bool ok = true;
        for (int j = x.first; j < x.end; ++j) {
          ok = mbar_wait_role(&s_full[t], (s_phase + j) & 1, abort);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[kTile];
#pragma unroll
          for (int b = 0; b < 4; ++b) tmem_ld32(s_at + 32 * b, s + 32 * b);
          tmem_wait_ld();
          if (j >= x.whole) {
            const int left = seen - j * kTile;  // keys of this tile the row sees
#pragma unroll
            for (int y = 0; y < kTile; ++y)
              if (y >= left) s[y] = 0xff800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int z = 0; z < kTile; z += 4)
#pragma unroll
            for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], __uint_as_float(s[z + y]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          if (j == x.first) {
            ref = top > -INFINITY ? top : kRefStart;
          } else {
            const bool raise = top > ref + kLazy;
            if (__any_sync(kFull, raise)) {
              // P V of the earlier tiles is done: S of this tile was issued behind it
              const float f = raise ? ex2(ref - top) : 1.f;
              if (raise) ref = top;
              part[0] = mul2(part[0], pair(f, f));
              part[1] = mul2(part[1], pair(f, f));
#pragma unroll 1
              for (int b = 0; b < DP / 32; ++b) {
                uint32_t o[32];
                tmem_ld32(o_at + 32 * b, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tmem_st32(o_at + 32 * b, o);
              }
            }
          }
          // 2^(c s - ref) two at a time; half of the weights go to the matrix unit while the other
          // half is computed
          const uint64_t c2 = pair(c, c), r2 = pair(-ref, -ref);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t p[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              float e0, e1;
              unpair(fma2(pair(__uint_as_float(s[32 * b + 2 * y]), __uint_as_float(s[32 * b + 2 * y + 1])),
                          c2, r2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              part[y & 1] = add2(part[y & 1], pair(e0, e1));
              p[y] = pack_bf16(e0, e1);
            }
            tmem_st16(s_at + 16 * b, p);
            if (b & 1) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[2 * t + (b >> 1)]);
            }
          }
        }
        s_phase += x.end;
        float sum;
        {
          float a0, a1, b0, b1;
          unpair(part[0], a0, a1);
          unpair(part[1], b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        }
        // ------------------------------------------------------------ epilogue
        if (ok) ok = __all_sync(kFull, mbar_wait_role(&o_full[t], o_phase, abort));
        o_phase ^= 1;
        if (ok) ok = __all_sync(kFull, mbar_wait_role(scrubbed, done & 1, abort));
        // a split's accumulators go where the other tile's products may still read K and V
        if (kSplit && ok && x.parts > 1 && x.two) ok = __all_sync(kFull, mbar_wait_role(&o_full[1], 0, abort));
        if (!kSplit && !ok) break;
        if (ok) {
          tc_fence_after();
          const bool check = *any_bad != 0;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key seen: zeros
          // 4 lanes hold 4 rows; they exchange 16-byte pieces, so that a store writes 64 bytes of
          // each of 8 rows (a row a lane, 16 bytes of 32 rows at a time, took 2 us a pair)
          __nv_bfloat16* out =
              a.out + ((int64_t)(x.q0 + x.t0 + t * a.tq) * a.q_heads + x.head * a.group) * a.head_dim +
              8 * (lane & 3);
          const int own = mine ? (tok * a.q_heads + g) * a.head_dim : -1;
          int to[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) to[y] = __shfl_sync(kFull, own, (lane & 28) + y);
#pragma unroll 1
          for (int b = 0; b < DP / 32; ++b) {
            uint32_t o[32];
            tmem_ld32(o_at + 32 * b, o);
            tmem_wait_ld();
            if (check) {
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (seen > bad[32 * b + y]) o[y] = 0x7fc00000u;
            }
            if (kSplit && x.parts > 1) {  // 16-byte piece y of a row at (y + row): no bank twice in 8 rows
              float4* to = reinterpret_cast<float4*>(smem) + (t * kTile + row) * (DP / 4);
#pragma unroll
              for (int y = 0; y < 8; ++y)
                to[(8 * b + y + row) & (DP / 4 - 1)] =
                    make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
              continue;
            }
            uint4 z[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t* e = o + 8 * y;
              auto two = [&](int k) { return pack_bf16(__uint_as_float(e[k]) * inv, __uint_as_float(e[k + 1]) * inv); };
              z[y] = make_uint4(two(0), two(2), two(4), two(6));
            }
#pragma unroll
            for (int m = 1; m < 4; m <<= 1) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                if (y & m) continue;
                exchange(z[y], z[y + m], lane & m, m);
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (to[y] >= 0 && 32 * b + 8 * (lane & 3) < a.head_dim)
                *reinterpret_cast<uint4*>(out + to[y] + 32 * b) = z[y];
          }
          if (kSplit && x.parts > 1)
            reinterpret_cast<float2*>(smem + L::kStats)[t * kTile + row] = make_float2(ref, sum);
        }
        // each tile for itself: the warps of a tile without work would be items ahead
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&written[t]);
      }
      done += work;
      w = following(item);
    }
    roles_met();
    if constexpr (kSplit) {
      // -------------------------------------------------------------- join of a split
      const Item x(read(0), a, split, rank_in);
      cluster_sync();
      if (x.parts > 1 && x.m > 0) {
        // rows rank_in, rank_in + CTAs, .., B to a warp at a time, 4 channels to a lane; all of
        // their parts are asked for (a far read takes about 0.5 us) before the first is used
        const int rows = x.two ? 2 * kTile : kTile;
        const int piece = lane & (DP / 4 - 1);
        auto join = [&](auto at_once) {
          constexpr int B = decltype(at_once)::value, C = kSplitMax / B;
          for (int x0 = warp; x0 * a.split + rank_in < rows; x0 += 8 * B) {
            float2 rs[B][C];
            float4 o[B][C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const uint32_t base = cluster_addr(smem, min(c, x.parts - 1));
#pragma unroll
              for (int b = 0; b < B; ++b) {
                const int at = (x0 + 8 * b) * a.split + rank_in;
                rs[b][c] = make_float2(kRefStart, 0.f);
                o[b][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < x.parts && at < rows) {
                  rs[b][c] = cluster_ld2(base + L::kStats + at * 8);
                  o[b][c] = cluster_ld4(base + (at * (DP / 4) + ((piece + at) & (DP / 4 - 1))) * 16);
                }
              }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
              const int at = (x0 + 8 * b) * a.split + rank_in;
              const int row = at & (kTile - 1), tok = row / a.group, g = row - tok * a.group;
              const int i = x.t0 + (at >> 7) * a.tq + tok;
              if (at >= rows || tok >= a.tq || i >= x.m) continue;
              float top = rs[b][0].x;
#pragma unroll
              for (int c = 1; c < C; ++c) top = fmaxf(top, rs[b][c].x);
              float sum = 0.f;
              uint64_t y[2] = {};
#pragma unroll
              for (int c = 0; c < C; ++c) {  // absent parts: nothing times at most 1
                const float f = ex2(rs[b][c].x - top);
                sum = fmaf(f, rs[b][c].y, sum);
                y[0] = fma2(pair(f, f), pair(o[b][c].x, o[b][c].y), y[0]);
                y[1] = fma2(pair(f, f), pair(o[b][c].z, o[b][c].w), y[1]);
              }
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              float z[4];
              unpair(y[0], z[0], z[1]);
              unpair(y[1], z[2], z[3]);
              if (lane < DP / 4 && 4 * piece < a.head_dim)
                *reinterpret_cast<uint2*>(
                    a.out + ((int64_t)(x.q0 + i) * a.q_heads + x.head * a.group + g) * a.head_dim + 4 * piece) =
                    make_uint2(pack_bf16(z[0] * inv, z[1] * inv), pack_bf16(z[2] * inv, z[3] * inv));
            }
          }
        };
        if (x.parts > 4) join(std::integral_constant<int, 1>{});
        else join(std::integral_constant<int, 4>{});
      }
      cluster_sync();  // no CTA ends while another reads its shared memory
    }
  }
  if (warp == 9) {
    tmem_dealloc(tmem, 512);
    if (lane == 0 && *abort != 0 && a.err != nullptr) atomicOr(a.err, KV_ERR_TIMEOUT);
  }
}

// How many clusters of each size run at once on the current device: the SMs come in groups of
// 16 to 20, of which a cluster takes its CTAs (152 SMs hold fewer than 19 clusters of 8).
template <int DP>
int clusters_at_once(int size) {
  static std::mutex mu;
  static int cached[64][kSplitMax + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& n = cached[dev][size];
  if (n == 0) {
    auto kernel = prompt_kernel<DP, kClusters, false>;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<DP>::kBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int found = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem<DP>::kBytes) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&found, kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    n = found > 0 ? found : -1;
  }
  return n;
}

// CTAs of a cluster: as many as let all `pairs` run at once and would have kSplitTiles each in a
// request that had all of the keys.
template <int DP>
int choose_split(int64_t pairs, int64_t keys) {
  const int64_t tiles = (keys + kTile - 1) / kTile;
  if (tiles < kSplitFrom || 2 * pairs > sm_count()) return 1;
  int64_t split = tiles / kSplitTiles < kSplitMax ? tiles / kSplitTiles : kSplitMax;
  if (split > sm_count() / pairs) split = sm_count() / pairs;
  while (split > 1 && clusters_at_once<DP>((int)split) < pairs) --split;
  return (int)split;
}

template <int DP, Mode kMode, bool kStall>
int launch(const PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
           cudaStream_t stream) {
  auto kernel = prompt_kernel<DP, kMode, kStall>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<DP>::kBytes) != cudaSuccess)
    return KV_ECUDA;
  if (kMode == kClusters &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                    cudaSuccess)
    return KV_ECUDA;
  const int64_t ctas = (int64_t)a.items * a.kv_heads * a.split;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  return launch_pdl_clusters(kernel, (unsigned)ctas, (unsigned)a.split, kThreads,
                             Smem<DP>::kBytes, stream, q, k, v, a);
}

template <int DP, bool kStall = false>
int launch(PromptArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
           cudaStream_t stream) {
  a.split = choose_split<DP>((int64_t)a.items * a.kv_heads, a.nk);
  if (a.split > 1) return launch<DP, kClusters, kStall>(a, q, k, v, stream);
  return (int64_t)a.items * a.kv_heads > sm_count()
             ? launch<DP, kManyWaves, kStall>(a, q, k, v, stream)
             : launch<DP, kOneWave, kStall>(a, q, k, v, stream);
}

// kStall: the self-test, with `stall_*` as in PromptArgs.
template <bool kStall>
int prompt(const void* query, int64_t query_stride, const void* key, int64_t key_stride,
           const void* value, int64_t value_stride, const int32_t* q_start_loc,
           const int32_t* k_start_loc, int32_t num_reqs, int32_t num_q_tokens, int32_t num_k_tokens,
           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale, void* out,
           int32_t* d_err, int32_t stall_role, int32_t stall_item, int64_t stall_ns,
           kv_stream_t stream) {
  if (num_reqs < 0 || num_q_tokens < 0 || num_k_tokens < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || num_q_heads % num_kv_heads != 0 ||
      !(scale > 0.f) || !(scale < INFINITY))
    return KV_EINVAL;
  if (head_dim % 8 != 0 || head_dim > 128 || num_q_heads / num_kv_heads > 128 ||
      num_q_heads > 4096 || num_reqs > KV_MAX_GATHER_REQS || num_q_tokens > KV_MAX_TOKENS ||
      num_k_tokens > KV_MAX_TOKENS)
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
                            overlap(out, out_bytes, value, (n1 * value_stride + k_row) * 2))) ||
      overlap(out, out_bytes, q_start_loc, (int64_t)(num_reqs + 1) * 4) ||
      overlap(out, out_bytes, k_start_loc, (int64_t)(num_reqs + 1) * 4))
    return KV_EINVAL;
  const int group = num_q_heads / num_kv_heads, tq = kTile / group;
  CUtensorMap q_map, k_map, v_map;
  // no key at all: nothing is loaded through the K and V maps
  const bool keys = num_k_tokens > 0;
  if (!rows_map(&q_map, query, query_stride, num_q_tokens, num_q_heads, head_dim, group, tq) ||
      !rows_map(&k_map, keys ? key : query, keys ? key_stride : query_stride,
                keys ? num_k_tokens : num_q_tokens, keys ? num_kv_heads : num_q_heads, head_dim, 1,
                kTile) ||
      !rows_map(&v_map, keys ? value : query, keys ? value_stride : query_stride,
                keys ? num_k_tokens : num_q_tokens, keys ? num_kv_heads : num_q_heads, head_dim, 1,
                kTile))
    return KV_ECUDA;
  // sum of ceil(m_r / pair) over the requests with a row, of which there are `some` at most
  const int some = num_reqs < num_q_tokens ? num_reqs : num_q_tokens;
  const int64_t items = (int64_t)(num_q_tokens - some) / (2 * tq) + some;
  // A single request has no others to be ranked with, and where its K and V are more than the L2
  // can be trusted with beside what else passes through it, its heads follow one another, so that one
  // head's K and V serve all CTAs at a time: 5.44 against 5.56 ms at 32768 tokens (134 MB), the same
  // at 12288 (50 MB); 111 against 92 us at 4096, where the longest pairs of all heads first count.
  const bool by_head = num_reqs == 1 && num_k_tokens * k_row * 4 > (int64_t)kL2Share;
  PromptArgs a{q_start_loc, k_start_loc, num_reqs, num_q_tokens, num_k_tokens, num_q_heads,
               num_kv_heads, head_dim, group, tq, (int32_t)items, 1, by_head,
               fminf(scale * 1.44269504088896340736f, FLT_MAX), static_cast<__nv_bfloat16*>(out), d_err,
               stall_role, stall_item, stall_ns};
  if constexpr (kStall) return launch<128, true>(a, q_map, k_map, v_map, stream);
  return head_dim <= 64 ? launch<64>(a, q_map, k_map, v_map, stream)
                        : launch<128>(a, q_map, k_map, v_map, stream);
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
  return prompt<false>(query, query_stride, key, key_stride, value, value_stride, q_start_loc,
                       k_start_loc, num_reqs, num_q_tokens, num_k_tokens, num_q_heads, num_kv_heads,
                       head_dim, scale, out, d_err, -1, 0, 0, stream);
}

extern "C" int kv_diag_attention_prompt_stall(
    const void* query, int64_t query_stride, const void* key, int64_t key_stride, const void* value,
    int64_t value_stride, const int32_t* q_start_loc, const int32_t* k_start_loc, int32_t num_reqs,
    int32_t num_q_tokens, int32_t num_k_tokens, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, float scale, void* out, int32_t* d_err, int32_t role, int32_t item,
    int64_t limit_ns, kv_stream_t stream) {
  if (role < 0 || role > kSoftmax + 1 || item < 0 || limit_ns < 0 ||
      limit_ns > (int64_t)kWaitLimitNs || d_err == nullptr)
    return KV_EINVAL;
  return prompt<true>(query, query_stride, key, key_stride, value, value_stride, q_start_loc,
                      k_start_loc, num_reqs, num_q_tokens, num_k_tokens, num_q_heads, num_kv_heads,
                      head_dim, scale, out, d_err, role, item, limit_ns, stream);
}
