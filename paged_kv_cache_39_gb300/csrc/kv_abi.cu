// kv_abi.cu -- status strings, ABI version and the per-device SM count.
#include <mutex>

#include "kv_tc.cuh"

namespace kvp {

int sm_count() {
  static std::mutex mu;
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 152;
    cached[dev] = n;
  }
  return cached[dev];
}

bool rows_map(CUtensorMap* map, const void* rows, int64_t stride, int64_t tokens, int heads,
              int head_dim, int box_heads, int box_tokens) {
  // the driver's entry point, asked for through the runtime: the library does not link libcuda
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows), dims, strides,
                box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvp

namespace kvp {
namespace {

// A wait that nothing will satisfy: an mbarrier expecting one arrival that
// never comes, waited on with the library's bounded wait.  It must give up
// after `limit` tries and report KV_ERR_TIMEOUT, leaving the context usable.
__global__ void bounded_wait_probe_kernel(int64_t limit, int32_t* err) {
  __shared__ uint64_t bar;
  if (threadIdx.x != 0) return;
  mbar_init(&bar, 1);
  mbar_fence_init();
  if (!mbar_wait_bounded(&bar, 0u, limit)) atomicOr(err, KV_ERR_TIMEOUT);
}

// The same with the wait that the prompt attention's roles share: warp w waits for a barrier of
// its own that never completes.  The first to give up makes the others leave.
__global__ void role_wait_probe_kernel(int64_t limit_ns, int64_t* waited_ns, int32_t* err) {
  __shared__ uint64_t bars[4];
  __shared__ int abort;
  if (threadIdx.x < 4) mbar_init(&bars[threadIdx.x], 1);
  if (threadIdx.x == 0) abort = 0;
  mbar_fence_init();
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const uint64_t t0 = global_ns();
  const bool ok = mbar_wait_role(&bars[warp], 0u, &abort, warp == 3 ? (uint64_t)limit_ns : kWaitLimitNs);
  if ((threadIdx.x & 31) == 0) waited_ns[warp] = (int64_t)(global_ns() - t0);
  if (!__any_sync(kFull, ok)) report(err, KV_ERR_TIMEOUT);
}

}  // namespace
}  // namespace kvp

extern "C" int kv_diag_role_wait(int64_t limit_ns, int64_t* d_waited_ns, int32_t* d_err,
                                 kv_stream_t stream) {
  if (limit_ns < 0 || limit_ns > (int64_t)kvp::kWaitLimitNs || d_waited_ns == nullptr ||
      !kvp::aligned(d_waited_ns, 8) || d_err == nullptr || !kvp::aligned(d_err, 4))
    return KV_EINVAL;
  kvp::role_wait_probe_kernel<<<1, 128, 0, stream>>>(limit_ns, d_waited_ns, d_err);
  return kvp::launch_status();
}

extern "C" int kv_diag_bounded_wait(int32_t spin_limit, int32_t* d_err, kv_stream_t stream) {
  if (spin_limit < 1 || spin_limit > (1 << 20) || d_err == nullptr ||
      !kvp::aligned(d_err, 4))
    return KV_EINVAL;
  kvp::bounded_wait_probe_kernel<<<1, 32, 0, stream>>>(spin_limit, d_err);
  return kvp::launch_status();
}

extern "C" const char* kv_status_string(int status) {
  switch (status) {
    case KV_OK: return "KV_OK";
    case KV_EINVAL: return "KV_EINVAL: invalid argument";
    case KV_EUNSUPPORTED: return "KV_EUNSUPPORTED: configuration rejected (fail closed)";
    case KV_ECUDA: return "KV_ECUDA: kernel launch failed";
    default: return "unknown kv_status";
  }
}

extern "C" int kv_abi_version(void) { return 7; }
