// kv_tc.cuh -- tcgen05 (matrix unit and tensor memory) and tiled-TMA helpers (sm_103a).
#pragma once

#include <cuda.h>

#include "kv_common.cuh"

namespace kvp {

// ---------------------------------------------------------------------------
// Tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(smem_dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define KVP_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define KVP_S4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
// 32 columns of this thread's lane (the warp's 32 lanes, one each).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVP_R4(r, 0), KVP_R4(r, 4), KVP_R4(r, 8), KVP_R4(r, 12), KVP_R4(r, 16), KVP_R4(r, 20),
        KVP_R4(r, 24), KVP_R4(r, 28)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      KVP_S4(r, 0), KVP_S4(r, 4), KVP_S4(r, 8), KVP_S4(r, 12), KVP_S4(r, 16), KVP_S4(r, 20),
      KVP_S4(r, 24), KVP_S4(r, 28)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      KVP_S4(r, 0), KVP_S4(r, 4), KVP_S4(r, 8), KVP_S4(r, 12)
      : "memory");
}
#undef KVP_R4
#undef KVP_S4

// True in one lane of a converged warp.  A role that issues for its CTA runs its loop and
// waits in the whole warp, so that the compiler keeps descriptors in uniform registers, and
// only the issue itself under this predicate (with the loop in one lane, every matrix
// instruction carried about 20 others and the issue, not the matrix unit, was the bound).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}

// ---------------------------------------------------------------------------
// Matrix instructions: D[128 x N] (+)= A[128 x 16] B[16 x N], bf16 in, fp32 out.

// Instruction descriptor: fp32 accumulator, bf16 operands; b_mn: B is stored with N contiguous.
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// Shared-memory operand of 128-byte rows in the 128-byte swizzle: 8-row groups are 1024
// bytes apart; `lead` is the distance of 64-element column blocks (N-contiguous operands).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(desc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrive on `bar` once every matrix instruction this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

// ---------------------------------------------------------------------------
// Barriers and tiled copies

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Wait for a phase, bounded like mbar_wait_bounded, but with no timer on the usual path: it
// starts after kUntimedTries (a try may suspend the thread for as long as the hardware likes, so
// only the timer bounds the time).  From then on every try is followed by a look at whether
// another role of the CTA has given up (*abort); one that gives up tells the others.
constexpr int kUntimedTries = 4;
__device__ __forceinline__ bool mbar_wait_role(uint64_t* bar, uint32_t parity, volatile int* abort,
                                               uint64_t limit_ns = kWaitLimitNs) {
#pragma unroll 1
  for (int i = 0; i < kUntimedTries; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (long i = 0; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort != 0) return false;
    if (global_ns() - t0 > limit_ns) break;
  }
  *abort = 1;
  return false;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------
// Clusters: every thread of every CTA arrives and waits; shared memory of CTA `rank`.

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void* mine, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(mine)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// Arithmetic of the softmax, and rows that change lanes

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

// ---------------------------------------------------------------------------
// Work stealing.  take_over() asks the hardware for a CTA of this grid that has not started (one
// thread; 16 bytes of answer, counted by `bar`, 16-byte aligned); if it gives one, that CTA never
// starts and its work is the asker's.  After a refusal no more is asked for.

__device__ __forceinline__ void take_over(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_addr(answer)),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ bool taken_over(const void* answer, int* block) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n .reg .b64 lo, hi;\n"
      " ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 h, {lo, hi};\n mov.u32 %1, 0;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
      : "=r"(ok), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  *block = (int)x;
  return ok != 0;
}

// Tensor map of bf16 rows [tokens, heads, head_dim] (`stride` elements between tokens) in boxes
// of 64 channels x box_heads x box_tokens, 128-byte swizzle, zeros outside.  False when the
// driver offers no encoder or refuses.
bool rows_map(CUtensorMap* map, const void* rows, int64_t stride, int64_t tokens, int heads,
              int head_dim, int box_heads, int box_tokens);

}  // namespace kvp
