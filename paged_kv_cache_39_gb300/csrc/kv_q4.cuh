// kv_q4.cuh -- the 4-bit paged cache: layout and addressing (sm_103a).
//
// A cache is [layers, blocks, kv_heads] records of block_size tokens.  A record
// holds the tokens' codes (head_dim / 2 bytes each), then their scales (one
// bf16 per 32 channels, head_dim / 16 bytes each), so the tokens of one
// (block, head) are contiguous and a reader of one head reads nothing else.
// With G = head_dim / 32, byte 2 G g + 2 j + b (g < 8, j < G, b < 2) of a
// token's codes holds channel 32 j + 4 g + 2 b in its low nibble and the next
// channel in its high one: a lane g of eight holds 4 channels of EVERY group,
// 2 G contiguous bytes.  A code c stands for (c - 8) * scale of its group.
#pragma once

#include <cuda_bf16.h>

#include "kv_common.cuh"

namespace kvp {

struct Q4Layout {
  int64_t layer_base;  // layer * num_blocks
  int64_t num_blocks;
  int32_t block_size, kv_heads, head_dim;

  __host__ __device__ __forceinline__ int64_t record_bytes() const {
    return (int64_t)block_size * (head_dim / 2 + head_dim / 16);
  }
  __device__ __forceinline__ int64_t record(int64_t block, int head) const {
    return ((layer_base + block) * kv_heads + head) * record_bytes();
  }
  // byte offsets inside a record
  __device__ __forceinline__ int64_t codes(int32_t token) const {
    return (int64_t)token * (head_dim / 2);
  }
  __device__ __forceinline__ int64_t scales(int32_t token) const {
    return (int64_t)block_size * (head_dim / 2) + (int64_t)token * (head_dim / 16);
  }
};

// Host-visible checks shared by the calls on a 4-bit cache.
inline int q4_checks(const void* k_cache, const void* v_cache, int32_t layer, int32_t num_layers,
                     int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                     int32_t head_dim, int32_t* d_err) {
  if (num_layers <= 0 || layer < 0 || layer >= num_layers || num_blocks < 1 || block_size <= 0 ||
      num_kv_heads <= 0 || head_dim <= 0)
    return KV_EINVAL;
  if (head_dim != 64 && head_dim != 128) return KV_EUNSUPPORTED;
  if (block_size % 8 != 0 || num_kv_heads > 4096) return KV_EUNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return KV_EINVAL;
  if (d_err != nullptr && !aligned(d_err, 4)) return KV_EINVAL;
  return KV_OK;
}

}  // namespace kvp
