// q8_writer.h -- launch interface of the block-scaled 8-bit cache's writer
// (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace smla {

struct Q8WriteParams {
  const __nv_bfloat16 *k, *v;      // [total][h_kv][d]
  int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  uint8_t *k_cache, *v_cache;      // [num_blocks][h_kv][64][d]
  int64_t k_block_bytes, v_block_bytes;
  float *k_scale, *v_scale;        // [num_blocks][h_kv]
  int64_t k_scale_stride, v_scale_stride, num_blocks;
  const int32_t* block_table;      // [batch][max_blocks]
  const int32_t* seqlens;          // [batch] before the new tokens
  const int32_t* new_seqlens;      // [batch] with them
  const int32_t* cu;               // [batch + 1]
  int max_blocks, batch, total, h_kv;
  uint32_t* status;                // may be NULL
};

cudaError_t launch_q8_write(const Q8WriteParams& p, int d, bool int8, cudaStream_t stream);

}  // namespace smla
