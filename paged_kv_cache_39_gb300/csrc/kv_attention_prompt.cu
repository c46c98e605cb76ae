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
//   8         TMA: Q once, then K and V tiles of 128 keys into a ring
//   9         issues the matrix instructions: S = Q K^T (both operands in shared
//             memory), O += P V (P from tensor memory, over the S it came from)
//   10, 11    check V tiles at the causal edge (below)
// While one tile's softmax runs, the matrix unit works for the other.  Tensor
// memory: S0 S1 (128 columns each, P in place), O0 O1: all 512 columns, hence one
// CTA per SM.
//
// Hidden keys.  A hidden logit is replaced, so a NaN there is gone, but 0 * NaN in
// P V is NaN.  So in the tiles where some key is hidden from some row (one to three
// per CTA), V values that are not finite are set to 0 in shared memory, and the
// first key that held one is kept per channel: rows that see that key
// get NaN in the epilogue.  Rows behind the sequence are set to 0 outright.
//
// Few rows behind many keys.  Where the tile pairs leave SMs idle, a cluster of up to 16 CTAs
// takes a pair, each CTA a run of its key tiles.  The CTAs then leave their accumulators, references
// and sums in their own shared memory, and each joins a share of the rows from all of them:
//   o_i = sum_c f_c O_c / sum_c f_c s_c,  f_c = 2^(ref_c - max ref).
// No workspace, no atomics: the same call gives the same bits.  The join costs 3 us; 16 tokens
// behind 8192 take 15 us instead of 74, behind 65536 58 instead of 558.
//
// Measured (32 query heads, 8 KV heads of 128 channels): one prompt of 32768 tokens 5.5 ms (1600
// TFLOP/s, at the card's power limit, 1.92 GHz), 16 chunks of 9 to 1855 tokens behind up to 7685
// 383 us (1310 TFLOP/s: the 7 CTAs that an SM runs one after another each take 4 us to start
// and to write, and the last wave is not full), 77 tokens 8.5 us.  Per 128 keys a CTA's two tiles
// take 3000 cycles: 2048 of matrix instructions; a tile's softmax is 1140, beside the other
// tile's products.
#include <cuda_bf16.h>

#include <mutex>
#include <type_traits>

#include "kv_tc.cuh"

namespace kvp {
namespace {

constexpr int kTile = 128;                 // query rows of a tile, keys of a K/V tile
constexpr int kThreads = 384;
constexpr int kScrubThreads = 64;
constexpr int kEdges = 3;                  // K/V tiles a CTA's rows see in part: 256 tokens span at most 3
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
  float scale_log2;
  __nv_bfloat16* out;
  int32_t* err;
};

template <int DP>
struct Smem {
  static constexpr int kTileBytes = kTile * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBars = kRing + kSlots * kTileBytes;
  // an edge tile's slot is not used again (it would have to be kSlots loads later)
  static_assert(kSlots >= 2 * kEdges - 1, "");
  // full[slots], empty[slots], edge[3], v_ok[3], q_full, s_full[2], p_full[2][2], o_full[2],
  // scrubbed, drain
  static constexpr int kNumBars = 2 * kSlots + 2 * kEdges + 11;
  static constexpr int kBad = kBars + kNumBars * 8;         // int[DP]: first key not finite
  static constexpr int kMisc = kBad + DP * 4;
  static constexpr int kBytes = kMisc + 64 + 1024;          // + alignment of the base
  // for the join of a split: fp32 accumulators and (reference, sum) of 2 x 128 rows, where Q, K
  // and V were
  static constexpr int kStats = 2 * kTile * DP * 4;
  static_assert(kStats + 2 * kTile * 8 <= kBars, "");
};

struct Work {
  int32_t q0, k0, m, n;  // the request's first rows and lengths
  int32_t t0;            // first token of the pair of tiles
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

// kSplit: in clusters of `split` CTAs (a kernel of its own, so that the other has neither the
// join's registers nor its code in its way: 5.46 against 5.63 ms at 32768 tokens).
template <int DP, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map, PromptArgs a) {
  using L = Smem<DP>;
  extern __shared__ unsigned char raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* full = bars;
  uint64_t* empty = full + L::kSlots;
  uint64_t* edge = empty + L::kSlots;
  uint64_t* v_ok = edge + kEdges;
  uint64_t* q_full = v_ok + kEdges;
  uint64_t* s_full = q_full + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 4;
  uint64_t* scrubbed = o_full + 2;
  uint64_t* drain = scrubbed + 1;
  int* bad = reinterpret_cast<int*>(smem + L::kBad);
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  int* any_bad = misc + 2;
  Work* s_work = reinterpret_cast<Work*>(misc + 4);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform for the compiler, too

  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kEdges; ++i) {
      mbar_init(&edge[i], 1);
      mbar_init(&v_ok[i], kScrubThreads);
    }
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], kTile / 32);  // the first 64 keys' weights, one arrival a warp
      mbar_init(&p_full[2 * i + 1], kTile / 32);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(scrubbed, kScrubThreads);
    mbar_init(drain, 1);
    mbar_fence_init();
    *abort = 0;
    *any_bad = 0;
    *s_work = Work{0, 0, 0, 0, 0};  // of a CTA that no pair is left for
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
  // A single request has no others to be ranked with: its heads follow one another instead, so
  // that one head's K and V (16.8 MB at 32768 tokens) serve all CTAs at a time (5.60 against
  // 5.66 ms).
  const bool single = a.num_reqs == 1;
  const int block = kSplit ? (int)(blockIdx.x / (unsigned)a.split) : (int)blockIdx.x;
  const int rank_in = kSplit ? (int)blockIdx.x - block * a.split : 0;
  const int head = single ? block / a.items : block % a.kv_heads;
  const int want = single ? block % a.items : block / a.kv_heads;
  uint32_t err = 0;
  {
    __shared__ int64_t warp_sum[kThreads / 32];
    int* keys_of = reinterpret_cast<int*>(smem);                     // [num_reqs], and
    int4* ranked = reinterpret_cast<int4*>(smem + kThreads * sizeof(int));  // the same: where Q will be
    const int pair = 2 * a.tq;
    const bool rank = a.num_reqs > 1 && a.num_reqs <= kThreads;
    const int per = (a.num_reqs + kThreads - 1) / kThreads;
    const int r_lo = min(a.num_reqs, tid * per), r_hi = min(a.num_reqs, r_lo + per);
    auto describe = [&](int r) {  // request r, or one without rows where it is not valid
      const int q0 = a.q_start[r], q1 = a.q_start[r + 1], k0 = a.k_start[r], k1 = a.k_start[r + 1];
      const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.nq && k0 >= 0 && k1 >= k0 && k1 <= a.nk;
      if (!ok) err |= KV_ERR_BAD_QSL;
      return ok ? Work{q0, k0, q1 - q0, k1 - k0, 0} : Work{0, 0, 0, 0, 0};
    };
    auto pairs = [&](const Work& x) { return (int)(((int64_t)x.m + pair - 1) / pair); };
    Work mine = {0, 0, 0, 0, 0};  // with `rank`: the request of this thread's rank
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
      }
      __syncthreads();
      if (tid < a.num_reqs) {
        const int4 x = ranked[tid];
        mine = Work{x.x, x.y, x.z, x.w, 0};
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
      mine.t0 = (pairs(mine) - 1 - (int)(want - at)) * pair;
      *s_work = mine;
    }
    __syncthreads();
    if (blockIdx.x == 0) report(a.err, err);
  }
  Work w = *s_work;  // the same in every lane: tell the compiler
  w.q0 = __shfl_sync(kFull, w.q0, 0);
  w.k0 = __shfl_sync(kFull, w.k0, 0);
  w.m = __shfl_sync(kFull, w.m, 0);
  w.n = __shfl_sync(kFull, w.n, 0);
  w.t0 = __shfl_sync(kFull, w.t0, 0);
  const int ahead = w.n - w.m;                                    // keys before the first query's own
  const int last = min(w.t0 + 2 * a.tq, w.m) - 1;                 // last token here
  const int keys = max(0, min(w.n, ahead + last + 1));            // keys the last token sees
  const int tiles = (keys + kTile - 1) / kTile;
  // this CTA's share of them: [first, end)
  const int parts = kSplit && tiles >= kSplitFrom ? min(a.split, tiles / kSplitTiles) : 1;
  const int first = kSplit && rank_in < parts ? tiles * rank_in / parts : 0;
  const int end = !kSplit ? tiles : rank_in < parts ? tiles * (rank_in + 1) / parts : 0;
  const int whole = max(0, ahead + w.t0 + 1) / kTile;             // tiles every row sees whole
  const bool two = w.t0 + a.tq < w.m;
  const bool work = w.m > 0 && end > first;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_ptr, 0);

  if (w.m > 0 && tiles == 0 && rank_in == 0) {  // no query here sees a key
    const int64_t row = (int64_t)a.group * a.head_dim;
    const int vecs = (int)(row / 8);
    for (int64_t i = tid; i < (int64_t)(last + 1 - w.t0) * vecs; i += kThreads) {
      const int64_t t = w.q0 + w.t0 + i / vecs;
      reinterpret_cast<uint4*>(a.out + t * a.q_heads * a.head_dim + head * row)[i % vecs] =
          make_uint4(0, 0, 0, 0);
    }
  }

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 && work) {
      // -------------------------------------------------------------- TMA
      const bool leader = elect_one();
      if (leader) {
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
        const uint32_t q_bytes = (uint32_t)(a.group * a.tq) * 128u * (DP / 64);
        mbar_arrive_expect_tx(q_full, two ? 2 * q_bytes : q_bytes);
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int c = 0; c < DP / 64; ++c)
            tma_load_3d(smem + L::kQ + t * L::kTileBytes + c * (kTile * 128), &q_map, 64 * c,
                        head * a.group, w.q0 + w.t0 + t * a.tq, q_full);
      }
      int u = 0, slot = 0, turn = 0;  // K and V tiles alternate in the ring
#pragma unroll 1
      for (; u < 2 * (end - first); ++u) {
        if (turn > 0 && !mbar_wait_role(&empty[slot], (turn - 1) & 1, abort)) break;
        const bool is_v = u & 1;
        const int j = first + (u >> 1);
        uint64_t* bar = is_v && j >= whole ? &edge[j - whole] : &full[slot];
        if (leader) {
          mbar_arrive_expect_tx(bar, L::kTileBytes);
          for (int c = 0; c < DP / 64; ++c)
            tma_load_3d(smem + L::kRing + slot * L::kTileBytes + c * (kTile * 128),
                        is_v ? &v_map : &k_map, 64 * c, head, w.k0 + j * kTile, bar);
        }
        if (++slot == L::kSlots) {
          slot = 0;
          ++turn;
        }
      }
      if (*abort != 0) {  // bounded wait for the copies still in flight
        mbar_wait_bounded(q_full, 0);
        for (int x = max(0, u - L::kSlots); x < u; ++x) {
          if ((x & 1) && first + (x >> 1) >= whole) mbar_wait_bounded(&edge[first + (x >> 1) - whole], 0);
          else mbar_wait_bounded(&full[x % L::kSlots], (x / L::kSlots) & 1);
        }
      }
    } else if (warp == 9 && work) {
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
      const int nt = two ? 2 : 1;
      bool ok = mbar_wait_role(q_full, 0, abort) && mbar_wait_role(&full[0], 0, abort);
      if (ok) {
        tc_fence_after();
        scores(0, 0);
        if (two) scores(1, 0);
        if (leader) mma_commit(&empty[0]);
      }
      int sv = 1, sk = 2, pv = 0, pk = 0;  // slots of V_j and K_{j+1}, parities of their phases
#pragma unroll 1
      for (int j = first; ok && j < end; ++j) {
        const bool more = j + 1 < end;
        const uint32_t phase = (j - first) & 1;
        // at the causal edge V is waited for through the warps that check it
        ok = j < whole ? mbar_wait_role(&full[sv], pv, abort)
                       : mbar_wait_role(&v_ok[j - whole], 0, abort);
        if (ok && more) ok = mbar_wait_role(&full[sk], pk, abort);
#pragma unroll 1
        for (int t = 0; ok && t < nt; ++t) {
          ok = mbar_wait_role(&p_full[2 * t], phase, abort);
          if (!ok) break;
          tc_fence_after();
          values(t, sv, j > first, 0);
          ok = mbar_wait_role(&p_full[2 * t + 1], phase, abort);
          if (!ok) break;
          tc_fence_after();
          values(t, sv, true, 1);
          if (more) scores(t, sk);  // in issue order behind the P V that reads what it overwrites
          else if (leader) mma_commit(&o_full[t]);
        }
        if (!ok) break;
        if (leader) {
          mma_commit(&empty[sv]);
          if (more) mma_commit(&empty[sk]);
        }
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
      }
      if (!ok) {  // bounded wait for the matrix instructions in flight
        if (leader) mma_commit(drain);
        mbar_wait_bounded(drain, 0);
      }
    } else if (warp >= 10 && work) {
      // -------------------------------------------------------------- V at the causal edge
      const int st = tid - 10 * 32;
      for (int j = max(first, whole); j < end; ++j) {
        const int slot = (2 * (j - first) + 1) % L::kSlots;
        if (!mbar_wait_role(&edge[j - whole], 0, abort)) break;
        unsigned char* tile = smem + L::kRing + slot * L::kTileBytes;
#pragma unroll 1
        for (int r = st; r < kTile; r += kScrubThreads) {
          const int key = j * kTile + r;
          // the row's 16-byte pieces, the row's own one first: no two of 8 rows share a bank
          auto piece = [&](int i) {
            return reinterpret_cast<uint4*>(tile + (i / 8) * (kTile * 128) + r * 128 + ((i + r) & 7) * 16);
          };
          if (key >= w.n) {
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) *piece(i) = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint32_t most = 0;  // the largest magnitudes, two to a word; 0x7f80 and up: not finite
#pragma unroll
          for (int i = 0; i < DP / 8; ++i) {
            const uint4 x = *piece(i);
            most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                           __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
          }
          if ((most & 0xffffu) < 0x7f80u && most < 0x7f800000u) continue;
#pragma unroll 1
          for (int i = 0; i < DP / 8; ++i) {
            uint4 x = *piece(i);
            uint32_t* e = reinterpret_cast<uint32_t*>(&x);
            const int channel = (i / 8) * 64 + (((i + r) & 7) ^ (r & 7)) * 8;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if ((e[q] & 0x7f80u) == 0x7f80u) {
                atomicMin(&bad[channel + 2 * q], key);
                e[q] &= 0xffff0000u;
              }
              if ((e[q] & 0x7f800000u) == 0x7f800000u) {
                atomicMin(&bad[channel + 2 * q + 1], key);
                e[q] &= 0xffffu;
              }
            }
            *piece(i) = x;
          }
          *any_bad = 1;
        }
        fence_proxy_async_smem();
        mbar_arrive(&v_ok[j - whole]);
      }
      mbar_arrive(scrubbed);
    }
    if constexpr (kSplit) {  // the softmax warps' join
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;  // the tile
    if (work && (t == 0 || two)) {
      // -------------------------------------------------------------- softmax
      const int row = tid & 127;
      const int tok = row / a.group, g = row - tok * a.group;
      const int i = w.t0 + t * a.tq + tok;  // token in the request
      const bool mine = tok < a.tq && i < w.m;
      const int seen = min(w.n, ahead + i + 1);
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes, in bits 16..
      const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 2 * kTile + t * DP;
      const float c = a.scale_log2;
      float ref = 0.f;
      uint64_t part[2] = {0, 0};  // sums of weights, two by two
      bool ok = true;
      for (int j = first; j < end; ++j) {
        ok = mbar_wait_role(&s_full[t], (j - first) & 1, abort);
        ok = __all_sync(kFull, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[kTile];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld32(s_at + 32 * b, s + 32 * b);
        tmem_wait_ld();
        if (j >= whole) {
          const int left = seen - j * kTile;  // keys of this tile the row sees
#pragma unroll
          for (int x = 0; x < kTile; ++x)
            if (x >= left) s[x] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kTile; x += 4)
#pragma unroll
          for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], __uint_as_float(s[x + y]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        if (j == first) {
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
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
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
          for (int x = 0; x < 16; ++x) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(s[32 * b + 2 * x]), __uint_as_float(s[32 * b + 2 * x + 1])),
                        c2, r2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            part[x & 1] = add2(part[x & 1], pair(e0, e1));
            p[x] = pack_bf16(e0, e1);
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
      float sum;
      {
        float a0, a1, b0, b1;
        unpair(part[0], a0, a1);
        unpair(part[1], b0, b1);
        sum = (a0 + a1) + (b0 + b1);
      }
      // -------------------------------------------------------------- epilogue
      if (ok) ok = __all_sync(kFull, mbar_wait_role(&o_full[t], 0, abort));
      if (ok) ok = __all_sync(kFull, mbar_wait_role(scrubbed, 0, abort));
      // a split's accumulators go where the other tile's products may still read K and V
      if (ok && parts > 1 && two) ok = __all_sync(kFull, mbar_wait_role(&o_full[1], 0, abort));
      if (ok) {
        tc_fence_after();
        const bool check = *any_bad != 0;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key seen: zeros
        __nv_bfloat16* out = a.out + ((int64_t)(w.q0 + i) * a.q_heads + head * a.group + g) * a.head_dim;
#pragma unroll 1
        for (int b = 0; b < DP / 32; ++b) {
          uint32_t o[32];
          tmem_ld32(o_at + 32 * b, o);
          tmem_wait_ld();
          if (check) {
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (seen > bad[32 * b + x]) o[x] = 0x7fc00000u;
          }
          if (parts > 1) {  // 16-byte piece x of a row at (x + row): no bank twice in 8 rows
            float4* to = reinterpret_cast<float4*>(smem) + (t * kTile + row) * (DP / 4);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              to[(8 * b + x + row) & (DP / 4 - 1)] =
                  make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                              __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
            continue;
          }
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint4 y;
            y.x = pack_bf16(__uint_as_float(o[x]) * inv, __uint_as_float(o[x + 1]) * inv);
            y.y = pack_bf16(__uint_as_float(o[x + 2]) * inv, __uint_as_float(o[x + 3]) * inv);
            y.z = pack_bf16(__uint_as_float(o[x + 4]) * inv, __uint_as_float(o[x + 5]) * inv);
            y.w = pack_bf16(__uint_as_float(o[x + 6]) * inv, __uint_as_float(o[x + 7]) * inv);
            if (mine && 32 * b + x < a.head_dim)
              *reinterpret_cast<uint4*>(out + 32 * b + x) = y;
          }
        }
        if (parts > 1)
          reinterpret_cast<float2*>(smem + L::kStats)[t * kTile + row] = make_float2(ref, sum);
      }
    }
    if constexpr (kSplit) {
      // -------------------------------------------------------------- join of a split
      cluster_sync();
      if (parts > 1 && w.m > 0) {
        // rows rank_in, rank_in + CTAs, .., B to a warp at a time, 4 channels to a lane; all of
        // their parts are asked for (a far read takes about 0.5 us) before the first is used
        const int rows = two ? 2 * kTile : kTile;
        const int piece = lane & (DP / 4 - 1);
        auto join = [&](auto at_once) {
          constexpr int B = decltype(at_once)::value, C = kSplitMax / B;
          for (int x0 = warp; x0 * a.split + rank_in < rows; x0 += 8 * B) {
            float2 rs[B][C];
            float4 o[B][C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const uint32_t base = cluster_addr(smem, min(c, parts - 1));
#pragma unroll
              for (int b = 0; b < B; ++b) {
                const int x = (x0 + 8 * b) * a.split + rank_in;
                rs[b][c] = make_float2(kRefStart, 0.f);
                o[b][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < parts && x < rows) {
                  rs[b][c] = cluster_ld2(base + L::kStats + x * 8);
                  o[b][c] = cluster_ld4(base + (x * (DP / 4) + ((piece + x) & (DP / 4 - 1))) * 16);
                }
              }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
              const int x = (x0 + 8 * b) * a.split + rank_in;
              const int row = x & (kTile - 1), tok = row / a.group, g = row - tok * a.group;
              const int i = w.t0 + (x >> 7) * a.tq + tok;
              if (x >= rows || tok >= a.tq || i >= w.m) continue;
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
                    a.out + ((int64_t)(w.q0 + i) * a.q_heads + head * a.group + g) * a.head_dim + 4 * piece) =
                    make_uint2(pack_bf16(z[0] * inv, z[1] * inv), pack_bf16(z[2] * inv, z[3] * inv));
            }
          }
        };
        if (parts > 4) join(std::integral_constant<int, 1>{});
        else join(std::integral_constant<int, 4>{});
      }
      cluster_sync();  // no CTA ends while another reads its shared memory
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
    auto kernel = prompt_kernel<DP, true>;
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
      found = 0;
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

template <int DP, bool kSplit>
int launch(const PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
           cudaStream_t stream) {
  auto kernel = prompt_kernel<DP, kSplit>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<DP>::kBytes) != cudaSuccess)
    return KV_ECUDA;
  if (kSplit && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                    cudaSuccess)
    return KV_ECUDA;
  const int64_t ctas = (int64_t)a.items * a.kv_heads * a.split;
  if (ctas > INT32_MAX) return KV_EUNSUPPORTED;
  return launch_pdl_clusters(kernel, (unsigned)ctas, (unsigned)a.split, kThreads,
                             Smem<DP>::kBytes, stream, q, k, v, a);
}

template <int DP>
int launch(PromptArgs a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
           cudaStream_t stream) {
  a.split = choose_split<DP>((int64_t)a.items * a.kv_heads, a.nk);
  return a.split > 1 ? launch<DP, true>(a, q, k, v, stream) : launch<DP, false>(a, q, k, v, stream);
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
                            overlap(out, out_bytes, value, (n1 * value_stride + k_row) * 2))))
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
  PromptArgs a{q_start_loc, k_start_loc, num_reqs, num_q_tokens, num_k_tokens, num_q_heads,
               num_kv_heads, head_dim, group, tq, (int32_t)items, 1,
               scale * 1.44269504088896340736f, static_cast<__nv_bfloat16*>(out), d_err};
  return head_dim <= 64 ? launch<64>(a, q_map, k_map, v_map, stream)
                        : launch<128>(a, q_map, k_map, v_map, stream);
}
