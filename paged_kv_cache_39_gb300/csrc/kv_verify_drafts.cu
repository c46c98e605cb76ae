// kv_verify_drafts.cu -- drafted tokens kept or refused by the target's probabilities, and the
// token behind them.
//
// Mathematics.  At a row with probabilities p (target) and q (draft), s_0 = p, Z_0 = 1; a child
// with token x and number u is kept when u q(x) Z_j < s_j(x), else
//   s_(j+1) = max(s_j - Z_j q, 0),  Z_(j+1) = sum s_(j+1);
// without q (1 at x): s loses x, Z_(j+1) = Z_j - s_j(x).  Behind the last child the token is the
// first t with sum_(k <= t) s(k) > u_0 sum s.  Only one token's s is needed for a test, so whole
// rows are read (a pass) for the sums alone: one after each refusal with q, whose sums the
// last token also uses, one at the end otherwise.
//
// A sum of 10^5 fp32 terms in 32 bits would move the borders between tokens by 1e-7 of the whole,
// and which token a number falls on would hang on the order of the sum.  So weights are
// integers, multiples of 2^-45: with s = h + l (h fp32, l what h's roundings left),
//   t = 1 + h in fp32 is h to a multiple of 2^-23, its bits are that integer;
//   h - (t - 1) is exact and 2^-24 at most, l is at most 2^-25 (half a step of an h below 1): their sum
//   stays within 0.75 * 2^-23, so with 1.5 * 2^-22 added it lies in [2^-22, 2^-21), where bits count 2^-45.
// (1.5 * 2^-23 would leave +-2^-24 only.)  The last two sums' roundings are 2^-48 and 2^-46: less than one
// unit together.
// Four additions and two integer ones an element, no conversions, and 64-bit sums whose order
// does not matter.  p - q is exact as h + l (both are known to 24 bits and p > q); s_j - Z_j q
// carries Z_j and s_j in two fp32 each, 2^-46 of the whole.
//
// GPU shape.  A cluster of CTAs per request: all of them go down the tree alike from the same
// few loads, and each warp sums a contiguous run of the row, which all learn of through
// shared memory.  The CTA that owns the run in which the last token falls reads it once more, out of
// the L2.
//
// Measured: 256 chains of 2 to 6 rows, 131072 fp32 probabilities (224 MB) 43 us, 5.2 TB/s: a CTA's passes
// follow one another with 32 KB in flight, and of the 304 CTAs that can run at once there are 256, so 48 of 152
// SMs have one where the others have two.  64 trees of 5 to 25 rows, 100003 in bf16 (21 MB) 36 to 41 us: up to a dozen
// refusals one after another, each a pass over the rows out of the L2 and a meeting of the cluster.  One chain of
// 6 rows, 32000: 7.7 to 8.5 us.  Two vectors in flight a thread: 43 us, four 54 (the 256 chains).  Without draft
// probabilities, where a refusal needs no pass: 32, 14.6 and 7.8 us.  An element goes through every refusal before it
// again, so 63 of them at one row (100003 in bf16) take 2.3 ms, and 53 us without draft probabilities.
#include <cuda_bf16.h>

#include "kv_tc.cuh"
#include "kv_tree.cuh"

namespace kvp {
namespace {

constexpr int kClusterMax = 8;
constexpr int kThreadsPerSm = 1024;  // at 64 registers
constexpr float kLowBias = 0x1.8p-22f;
constexpr int kLowBits = 22;               // of a weight, in units: t's are 2^-23
constexpr double kUnit = 0x1p-45;

struct VerifyArgs {
  const void* target;
  int64_t target_stride;
  const void* draft;  // or null
  int64_t draft_stride;
  int32_t vocab;
  const int32_t* tokens;
  const int32_t* parents;  // or null
  const int32_t* q_start;
  const float* uniform;
  int32_t num_rows, cluster;
  int32_t* out_tokens;
  int32_t* path;
  int32_t* num_kept;
  int32_t* err;
};

__device__ __forceinline__ float value(float x) { return __saturatef(x); }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __saturatef(__bfloat162float(x)); }

// What a pass sums: p, p - q, or the s of several refusals.
enum Kind { kWhole, kFirst, kMore };

// s of 2 N elements as h + l, two in a register pair.  z: Z_1 .. Z_(count - 1) in two parts.
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }
__device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) { return fma2(y, both(-1.f), x); }
template <Kind kind, int N>
__device__ __forceinline__ void left_of(const float (&p)[2 * N], const float (&q)[2 * N], const float2* z,
                                        int count, uint64_t (&h)[N], uint64_t (&l)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t pp = pair(p[2 * i], p[2 * i + 1]);
    h[i] = pp;
    l[i] = 0;
    if constexpr (kind != kWhole) {
      // q no larger than p: the difference, and what its rounding leaves, are exact and not below 0
      const uint64_t qq = pair(fminf(q[2 * i], p[2 * i]), fminf(q[2 * i + 1], p[2 * i + 1]));
      h[i] = sub2(pp, qq);
      l[i] = sub2(sub2(pp, h[i]), qq);
    }
  }
  if constexpr (kind == kMore) {
#pragma unroll 1
    for (int j = 1; j < count; ++j) {
      const float2 zj = z[j];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t qq = pair(q[2 * i], q[2 * i + 1]);
        const uint64_t less = mul2(both(-zj.x), qq);                                // -Z q = less - more
        const uint64_t more = fma2(both(zj.y), qq, fma2(both(zj.x), qq, less));
        const uint64_t d = add2(h[i], less), back = sub2(d, h[i]);
        const uint64_t rest = add2(sub2(sub2(h[i], sub2(d, back)), sub2(back, less)), sub2(l[i], more));
        float x[2], y[2];
        h[i] = add2(d, rest);
        l[i] = sub2(rest, sub2(h[i], d));
        unpair(h[i], x[0], x[1]);
        unpair(l[i], y[0], y[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          y[e] = x[e] > 0.f ? y[e] : 0.f;
          x[e] = fmaxf(x[e], 0.f);
        }
        h[i] = pair(x[0], x[1]);
        l[i] = pair(y[0], y[1]);
      }
    }
  }
}
// The two integers of each s, biased: their sums are taken off again by count.
__device__ __forceinline__ void add_weights(uint64_t h, uint64_t l, uint32_t& hi, uint32_t& lo) {
  const uint64_t t = add2(h, both(1.f));
  const uint64_t low = add2(add2(sub2(h, add2(t, both(-1.f))), l), both(kLowBias));
  hi += (uint32_t)t + (uint32_t)(t >> 32);
  lo += (uint32_t)low + (uint32_t)(low >> 32);
}
__device__ __forceinline__ uint64_t weight_sum(uint32_t hi, uint32_t lo, uint32_t count) {
  hi -= count * 0x3f800000u;
  lo -= count * __float_as_uint(kLowBias);
  return ((uint64_t)hi << kLowBits) + (uint64_t)(int64_t)(int32_t)lo;
}
template <Kind kind>
__device__ __forceinline__ uint64_t weight_of(float p, float q, const float2* z, int count) {
  const float p2[2] = {p, 0.f}, q2[2] = {q, 0.f};
  uint64_t h[1], l[1];
  uint32_t hi = 0, lo = 0;
  left_of<kind, 1>(p2, q2, z, count, h, l);
  add_weights(h[0], l[0], hi, lo);
  return weight_sum(hi, lo, 2);  // the other one is 0
}

template <typename T>
struct Vec {
  static constexpr int kElems = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __saturatef(__uint_as_float(v.x));
  x[1] = __saturatef(__uint_as_float(v.y));
  x[2] = __saturatef(__uint_as_float(v.z));
  x[3] = __saturatef(__uint_as_float(v.w));
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __saturatef(__uint_as_float(w[k] << 16));
    x[2 * k + 1] = __saturatef(__uint_as_float(w[k] & 0xffff0000u));
  }
}

// A row of V elements cut into `parts` runs of whole 16-byte vectors; the first run has what lies before
// the first vector, the last one what lies behind the last.
template <typename T>
struct Cut {
  int head, vecs;
  bool vector;  // both rows have their vectors at the same elements
  __device__ __forceinline__ Cut(const T* p, const T* q, int V) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) & 15, b = reinterpret_cast<uintptr_t>(q) & 15;
    vector = q == nullptr || a == b;
    head = vector ? (int)(((16 - a) & 15) / sizeof(T)) : 0;
    if (head > V) head = V;
    vecs = vector ? (V - head) / Vec<T>::kElems : V;
  }
  // first vector (element, where there are none) of run g
  __device__ __forceinline__ int from(int g, int parts) const { return (int)((int64_t)vecs * g / parts); }
  __device__ __forceinline__ int element(int g, int parts, int V) const {
    if (g == 0) return 0;
    if (g == parts) return V;
    return head + from(g, parts) * (vector ? Vec<T>::kElems : 1);
  }
};

// Sum of the weights of run g, over a warp.
template <typename T, Kind kind>
__device__ uint64_t run_sum(const T* p, const T* q, int V, int g, int parts, const float2* z,
                            int count) {
  constexpr int E = Vec<T>::kElems, U = 2;  // vectors asked for at once
  const int lane = threadIdx.x & 31;
  const Cut<T> cut(p, kind == kWhole ? nullptr : q, V);
  uint64_t sum = 0;
  auto one = [&](int i) {
    sum += weight_of<kind>(value(p[i]), kind == kWhole ? 0.f : value(q[i]), z, count);
  };
  const int v0 = cut.from(g, parts), v1 = cut.from(g + 1, parts);
  if (!cut.vector) {
#pragma unroll 4
    for (int i = v0 + lane; i < v1; i += 32) one(i);
  } else {
    const uint4* pv = reinterpret_cast<const uint4*>(p + cut.head);
    const uint4* qv = reinterpret_cast<const uint4*>(q + (kind == kWhole ? 0 : cut.head));
    for (int v = v0 + lane; v < v1; v += 32 * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool in = v + 32 * k < v1;
        a[k] = in ? ld_stream(pv + v + 32 * k) : make_uint4(0, 0, 0, 0);
        if (kind != kWhole) b[k] = in ? ld_stream(qv + v + 32 * k) : make_uint4(0, 0, 0, 0);
      }
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float x[E], y[E];
        unpack(a[k], x);
        if (kind != kWhole) unpack(b[k], y);
        else unpack(make_uint4(0, 0, 0, 0), y);
        constexpr int N = kind == kMore ? E / 2 : 1;  // pairs at a time: more where they wait for one another's Z
#pragma unroll
        for (int e = 0; e < E; e += 2 * N) {
          float p2[2 * N], q2[2 * N];
          uint64_t h[N], l[N];
#pragma unroll
          for (int i = 0; i < 2 * N; ++i) p2[i] = x[e + i], q2[i] = y[e + i];
          left_of<kind, N>(p2, q2, z, count, h, l);
#pragma unroll
          for (int i = 0; i < N; ++i) add_weights(h[i], l[i], hi, lo);
        }
      }
      sum += weight_sum(hi, lo, U * E);
    }
    if (g == 0 && lane < cut.head) one(lane);
    const int tail = cut.head + cut.vecs * E;
    if (g == parts - 1 && tail + lane < V) one(tail + lane);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  return sum;
}

__device__ __forceinline__ void store_far(uint64_t* mine, int rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(mine, rank)), "l"(v) : "memory");
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreadsPerSm / kThreads) verify_kernel(VerifyArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ uint64_t s_sums[2][kClusterMax * kWarps];  // of the runs; passes take turns
  __shared__ uint64_t s_scan[kWarps];
  __shared__ int s_token[kTreeRows], s_parent[kTreeRows], s_path[kTreeRows];
  __shared__ float s_u[kTreeRows], s_p[kTreeRows], s_q[kTreeRows];
  __shared__ int s_gone[kTreeRows];                     // tokens that s lost (no q)
  __shared__ float2 s_z[kTreeRows + 1];
  __shared__ double s_zd[kTreeRows + 1];
  __shared__ int s_at, s_count, s_pass, s_kept, s_final, s_run;
  __shared__ uint64_t s_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / a.cluster, rank = blockIdx.x - r * a.cluster;
  pdl_allow_next();
  pdl_wait();
  const StepRows rows = step_rows(a.q_start, r, a.num_rows, kTreeRows);
  const int m = rows.count, V = a.vocab;
  if (m <= 0) {  // in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      a.num_kept[r] = 0;
      if (m < 0) report(a.err, KV_ERR_BAD_QSL);
    }
    return;
  }
  const T* const target = static_cast<const T*>(a.target) + (int64_t)rows.first * a.target_stride;
  const T* const draft = a.draft == nullptr
                             ? nullptr
                             : static_cast<const T*>(a.draft) + (int64_t)rows.first * a.draft_stride;
  // ---- every row's token, number and its own two probabilities
  if (tid < kTreeRows) {
    uint32_t err = 0;
    int parent = -2, token = -1;
    float p = 0.f, q = 1.f, u = 0.f;
    if (tid < m) {
      u = a.uniform[rows.first + tid];
      u = u < 0x1.fffffep-1f ? fmaxf(u, 0.f) : u >= 0x1.fffffep-1f ? 0x1.fffffep-1f : 0.f;
    }
    if (tid > 0 && tid < m) {
      token = a.tokens[rows.first + tid];
      parent = a.parents != nullptr ? a.parents[rows.first + tid] : tid - 1;
      if (token < 0 || token >= V) err |= KV_ERR_BAD_TOKEN;
      if (parent < 0 || parent >= tid) err |= KV_ERR_BAD_TREE;
      if (err != 0) {
        parent = -2;
      } else {
        p = value(target[parent * a.target_stride + token]);
        if (draft != nullptr) q = value(draft[parent * a.draft_stride + token]);
      }
    }
    s_token[tid] = token;
    s_parent[tid] = parent;
    s_u[tid] = u;
    s_p[tid] = p;
    s_q[tid] = q;
    if (rank == 0) report(a.err, err);
  }
  if (tid == 0) {
    s_path[0] = 0;
    s_zd[0] = 1.0;
  }
  // before the first far store: the other CTAs run
  if (a.cluster > 1) cluster_sync();
  __syncthreads();

  // ---- down the tree.  Thread 0 goes on until a whole row is needed (s_pass: 1 for Z, 2 for the
  // last token), all do that, and so on.
  const int parts = a.cluster * kWarps, g = rank * kWarps + warp;
  int row = 1, at = 0, kept = 0, count = 0;  // thread 0's: next row to try; where; refusals there
  bool known = false;                        // the sums of (at, count) are there
  uint64_t whole = 0;
  int turn = 0;
  // at most a pass for each row but the first, and two for the last token, whatever is read (counting them takes
  // a register too many: 256 chains 54 us instead of 43)
  while (true) {
    if (tid == 0) {
      int pass = 0;
      for (; row < m && pass == 0; ++row) {
        if (s_parent[row] != at) continue;
        const int token = s_token[row];
        double left = s_p[row], q = s_q[row];
        if (draft == nullptr) {
          for (int j = 0; j < count; ++j)
            if (s_gone[j] == token) left = 0.0;
        } else {
          for (int j = 0; j < count; ++j) left = fmax(left - s_zd[j] * q, 0.0);
        }
        if ((double)s_u[row] * q * s_zd[count] < left) {
          at = row;
          s_path[++kept] = row;
          count = 0;
          known = false;
        } else if (draft != nullptr) {
          ++count;
          pass = 1;
        } else if (left > 0.0 || count == 0) {  // a token that is gone already stays gone
          s_zd[count + 1] = fmax(s_zd[count] - left, 0.0);
          s_gone[count++] = token;
        }
      }
      if (pass == 0) {
        if (known && whole == 0 && count > 0) {  // nothing is left: p again
          count = 0;
          known = false;
        }
        pass = known ? 3 : 2;
      }
      s_at = at;
      s_count = count;
      s_pass = pass;
      s_kept = kept;
    }
    __syncthreads();
    const int pass = s_pass, n = s_count, here = s_at;
    if (pass == 3) break;
    // ---- a pass: every warp its run
    const T* p = target + here * a.target_stride;
    const T* q = draft == nullptr ? nullptr : draft + here * a.draft_stride;
    uint64_t sum;
    if (draft == nullptr || n == 0) {
      sum = run_sum<T, kWhole>(p, q, V, g, parts, s_z, n);
      if (n > 0) {  // without the tokens that are gone
        const Cut<T> cut(p, nullptr, V);
        const int lo = cut.element(g, parts, V), hi = cut.element(g + 1, parts, V);
        uint64_t off = 0;
        for (int j = lane; j < n; j += 32)
          if (s_gone[j] >= lo && s_gone[j] < hi)
            off += weight_of<kWhole>(value(p[s_gone[j]]), 0.f, s_z, 0);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) off += __shfl_xor_sync(kFull, off, d);
        sum -= off;
      }
    } else if (n == 1) {
      sum = run_sum<T, kFirst>(p, q, V, g, parts, s_z, n);
    } else {
      sum = run_sum<T, kMore>(p, q, V, g, parts, s_z, n);
    }
    if (a.cluster > 1) {
      if (lane < a.cluster) store_far(&s_sums[turn][g], lane, sum);
      cluster_sync();
    } else if (lane == 0) {
      s_sums[turn][g] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      whole = 0;
      for (int i = lane; i < parts; i += 32) whole += s_sums[turn][i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) whole += __shfl_xor_sync(kFull, whole, d);
    }
    if (tid == 0) {
      if (pass == 1) {
        const double z = (double)whole * kUnit;
        s_zd[n] = z;
        s_z[n] = make_float2((float)z, (float)(z - (double)(float)z));
      }
      known = true;
    }
    turn ^= 1;
  }
  // ---- the last token: the run it falls into, then the element
  const int n = s_count, here = s_at, n_kept = s_kept;
  const T* p = target + here * a.target_stride;
  const T* q = draft == nullptr ? nullptr : draft + here * a.draft_stride;
  if (warp == 0) {
    const uint64_t* sums = s_sums[turn ^ 1];
    const uint64_t want = (uint64_t)((double)s_u[0] * (double)whole);
    // runs lane * each .. of this lane, their sum and that of all up to them
    const int each = (parts + 31) / 32;
    uint64_t mine = 0;
    for (int i = lane * each; i < min(parts, (lane + 1) * each); ++i) mine += sums[i];
    const uint64_t incl = warp_inclusive_scan<uint64_t>(mine);
    const uint32_t past = __ballot_sync(kFull, incl > want);
    if (lane == (past != 0 ? __ffs(past) - 1 : 0)) {  // none: nothing has a weight
      uint64_t rest = want - (incl - mine);
      int run = lane * each;
      while (past != 0 && sums[run] <= rest) rest -= sums[run++];
      s_run = run;
      s_want = rest;
      s_final = -1;
    }
  }
  __syncthreads();
  const int run = s_run;
  const uint64_t want = s_want;
  if (run / kWarps != rank) return;
  // Its elements once more, a piece in a row for every thread; then the 32 lanes around the thread whose
  // piece it is take that one element by element.  Short code: it runs once, and waits for itself.
  const bool only_p = draft == nullptr || n == 0;
  const Cut<T> cut(p, only_p ? nullptr : q, V);
  const int lo = cut.element(run, parts, V), hi = cut.element(run + 1, parts, V);
  auto weight = [&](int i) {
    const float x = value(p[i]), y = only_p ? 0.f : value(q[i]);
    uint64_t w = only_p ? weight_of<kWhole>(x, y, s_z, 0) : weight_of<kMore>(x, y, s_z, n);
    if (draft == nullptr)
      for (int j = 0; j < n; ++j)
        if (s_gone[j] == i) w = 0;
    return w;
  };
  // [i0, i1): this thread's piece, of whole vectors but for what the run has before and behind them
  constexpr int E = Vec<T>::kElems, kAtOnce = 2;
  const int v0 = cut.from(run, parts), vecs = cut.from(run + 1, parts) - v0;
  const int each = (vecs + kThreads - 1) / kThreads, a0 = min(vecs, tid * each), a1 = min(vecs, a0 + each);
  const int size = cut.vector ? E : 1, body = cut.head + v0 * size;
  const int i0 = tid == 0 ? lo : body + a0 * size, i1 = tid == kThreads - 1 ? hi : body + a1 * size;
  uint64_t mine = 0;
  for (int i = i0; i < body; ++i) mine += weight(i);
  for (int i = body + vecs * size; i < i1; ++i) mine += weight(i);
  if (!cut.vector) {
#pragma unroll 4
    for (int i = body + a0; i < body + a1; ++i) mine += weight(i);
  } else {
    const uint4* pv = reinterpret_cast<const uint4*>(p + cut.head) + v0;
    const uint4* qv = only_p ? pv : reinterpret_cast<const uint4*>(q + cut.head) + v0;
    for (int v = a0; v < a1; v += kAtOnce) {
      uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const bool in = v + k < a1;
        x[k] = in ? pv[v + k] : make_uint4(0, 0, 0, 0);
        y[k] = in && !only_p ? qv[v + k] : make_uint4(0, 0, 0, 0);
      }
      uint32_t hi32 = 0, lo32 = 0;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        float f[E], g[E];
        uint64_t h[E / 2], l[E / 2];
        unpack(x[k], f);
        unpack(y[k], g);  // zeros leave p as it is
        left_of<kMore, E / 2>(f, g, s_z, only_p ? 0 : n, h, l);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) add_weights(h[e], l[e], hi32, lo32);
      }
      mine += weight_sum(hi32, lo32, kAtOnce * E);
    }
    if (draft == nullptr)
      for (int j = 0; j < n; ++j)
        if (s_gone[j] >= max(i0, body) && s_gone[j] < min(i1, body + vecs * size))
          mine -= weight_of<kWhole>(value(p[s_gone[j]]), 0.f, s_z, 0);
  }
  uint64_t incl = warp_inclusive_scan<uint64_t>(mine);
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) incl += s_scan[w];
  const uint32_t found = __ballot_sync(kFull, incl > want && incl - mine <= want);
  if (found != 0) {  // in this warp; in no warp where nothing has a weight
    const int src = __ffs(found) - 1;
    uint64_t up = __shfl_sync(kFull, incl - mine, src);
    const int from = __shfl_sync(kFull, i0, src), to = __shfl_sync(kFull, i1, src);
    // as far as the piece goes: it holds the token, unless its elements have changed since the first look
    for (int at_i = from; at_i < to; at_i += 32) {
      const int i = at_i + lane;
      const uint64_t w = warp_inclusive_scan<uint64_t>(i < to ? weight(i) : 0);
      const uint32_t past = __ballot_sync(kFull, up + w > want);
      if (past != 0) {
        if (lane == __ffs(past) - 1) s_final = i;
        break;
      }
      up += __shfl_sync(kFull, w, 31);
    }
  }
  __syncthreads();
  const int last = s_final;
  if (tid < m) {
    a.out_tokens[rows.first + tid] = tid < n_kept ? s_token[s_path[tid + 1]] : tid == n_kept ? last : -1;
    a.path[rows.first + tid] = tid <= n_kept ? s_path[tid] : -1;
  }
  if (tid == 0) {
    a.num_kept[r] = n_kept;
    if (last < 0) report(a.err, KV_ERR_BAD_PROBS);
  }
}

template <typename T, int kThreads>
int launch(const VerifyArgs& a, int32_t num_reqs, cudaStream_t stream) {
  return launch_pdl_clusters(verify_kernel<T, kThreads>, (unsigned)num_reqs * a.cluster, a.cluster,
                             kThreads, 0, stream, a);
}
// A request to a CTA where there are more of them than SMs, else as many smaller CTAs to each as run at
// once, 8 at most.  256 chains of 131072: 43 us so, 47 with two or four of 256 threads; 64 trees of
// 100003 in bf16: 36 us with 8 of 256 threads, 41 with 8 of 512, 44 with 4 of 512.
template <typename T>
int launch(VerifyArgs a, int32_t num_reqs, cudaStream_t stream) {
  a.cluster = 1;
  if (num_reqs > sm_count()) return launch<T, 512>(a, num_reqs, stream);
  while (a.cluster < kClusterMax && num_reqs * a.cluster * 2 <= kThreadsPerSm / 256 * sm_count())
    a.cluster *= 2;
  return launch<T, 256>(a, num_reqs, stream);
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_verify_drafts(const void* target_probs, int64_t target_stride,
                                const void* draft_probs, int64_t draft_stride, int32_t prob_type,
                                int32_t vocab, const int32_t* tokens, const int32_t* parents,
                                const int32_t* q_start_loc, const float* uniform,
                                int32_t num_reqs, int32_t num_rows, int32_t* out_tokens,
                                int32_t* path, int32_t* num_kept, int32_t* d_err,
                                kv_stream_t stream) {
  const int rc = step_checks(num_reqs, num_rows, d_err);
  if (rc != KV_OK) return rc;
  if (vocab < 1 || (prob_type != KV_F32 && prob_type != KV_BF16)) return KV_EINVAL;
  if (vocab > 1 << 20) return KV_EUNSUPPORTED;
  if (target_stride < vocab || (draft_probs != nullptr && draft_stride < vocab)) return KV_EINVAL;
  if (num_reqs == 0) return KV_OK;
  const int size = prob_type == KV_F32 ? 4 : 2;
  if (q_start_loc == nullptr || num_kept == nullptr || !aligned(q_start_loc, 4) ||
      !aligned(num_kept, 4))
    return KV_EINVAL;
  if (num_rows > 0 && (target_probs == nullptr || tokens == nullptr || uniform == nullptr ||
                       out_tokens == nullptr || path == nullptr))
    return KV_EINVAL;
  if (!aligned(target_probs, size) || !aligned(draft_probs, size) || !aligned(tokens, 4) ||
      !aligned(parents, 4) || !aligned(uniform, 4) || !aligned(out_tokens, 4) || !aligned(path, 4))
    return KV_EINVAL;
  const int64_t n4 = (int64_t)num_rows * 4, last = (int64_t)num_rows - 1;
  void* const outs[3] = {out_tokens, path, num_kept};
  const int64_t bytes[3] = {n4, n4, (int64_t)num_reqs * 4};
  for (int i = 0; i < 3; ++i) {
    const auto over = [&](const void* p, int64_t size_of) { return overlap(outs[i], bytes[i], p, size_of); };
    if (over(tokens, n4) || over(parents, n4) || over(uniform, n4) ||
        over(q_start_loc, (int64_t)(num_reqs + 1) * 4) ||
        over(outs[(i + 1) % 3], bytes[(i + 1) % 3]) ||
        (num_rows > 0 && (over(target_probs, (last * target_stride + vocab) * size) ||
                          over(draft_probs, (last * draft_stride + vocab) * size))))
      return KV_EINVAL;
  }
  const VerifyArgs a{target_probs, target_stride, draft_probs, draft_stride, vocab, tokens, parents,
                     q_start_loc, uniform, num_rows, 1, out_tokens, path, num_kept, d_err};
  return prob_type == KV_F32 ? launch<float>(a, num_reqs, stream)
                             : launch<__nv_bfloat16>(a, num_reqs, stream);
}
