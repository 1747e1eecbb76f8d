// block_table.cu -- block tables and slot maps of a serving step, built on the
// GPU from the requests' lengths.
//
// Request r holds len_r tokens in ceil(len_r / 64) blocks and takes new_r more:
//   need_r   = ceil((len_r + new_r) / 64) - ceil(len_r / 64)
//   first_r  = sum_{i < r} need_i,   cu_r = sum_{i < r} new_i
//   block ceil(len_r / 64) + i of request r = free[num_free - 1 - first_r - i]
//   slot of its token t: block of position len_r + t, times 64, plus the rest.
// A request whose blocks do not all fit keeps its length and gets slots -1; so does one
// whose length would pass 2^31 - 1.
//
// Bound by latency: the smallest step reads and writes a few KB.  Every CTA
// scans the lengths itself (one shuffle scan of tokens and blocks per 1024
// requests), so one launch does it all and no CTA waits
// for another; slots of fresh blocks come from the free list, never from table
// entries that another CTA may be writing.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smla.h"
#include "splitkv_mla.h"

namespace smla {

constexpr int kTableThreads = 1024;

// Blocks of len tokens, 0 <= len < 2^31.
__device__ __forceinline__ int blocks_of(int len) { return (int)(((uint32_t)len + 63u) / 64u); }

__global__ void __launch_bounds__(kTableThreads)
    extend_block_table_kernel(int32_t* block_table, int max_blocks, const int32_t* __restrict__ seqlens,
                              const int32_t* __restrict__ new_lens, int batch,
                              const int32_t* __restrict__ free_blocks, int64_t free_capacity,
                              const int32_t* __restrict__ num_free, int64_t max_new_tokens,
                              int64_t* __restrict__ slots, int32_t* __restrict__ cu_new,
                              int32_t* __restrict__ seqlens_out, int32_t* __restrict__ num_free_out) {
  __shared__ uint64_t warp_tokens[32], warp_blocks[32];
  __shared__ int64_t s_cu[kTableThreads + 1];   // first token of each request
  __shared__ int32_t s_len[kTableThreads], s_first[kTableThreads], s_need[kTableThreads];
  __shared__ int s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t have = min((int64_t)max(num_free[0], 0), free_capacity);
  // this CTA's tokens
  const int64_t per = (max_new_tokens + gridDim.x - 1) / gridDim.x;
  const int64_t i0 = min(per * blockIdx.x, max_new_tokens), i1 = min(i0 + per, max_new_tokens);
  int64_t tokens = 0, blocks = 0;               // before this chunk of requests
  if (tid == 0) s_taken = 0;
  for (int r0 = 0; r0 < batch; r0 += kTableThreads) {
    const int r = r0 + tid;
    int len = 0, fresh = 0, need = 0;
    if (r < batch) {
      len = max(seqlens[r], 0);
      fresh = max(new_lens[r], 0);
      const int64_t sum = (int64_t)len + fresh;
      const bool room = sum <= 0x7FFFFFFF && (sum + 63) / 64 <= max_blocks;
      need = room ? blocks_of((int)sum) - blocks_of(len) : -1;
    }
    uint64_t t64 = (uint64_t)fresh, b64 = (uint64_t)max(need, 0);   // inclusive sums of tokens and blocks
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, t64, off), z = __shfl_up_sync(0xffffffffu, b64, off);
      if (lane >= off) t64 += y, b64 += z;
    }
    __syncthreads();                            // the chunk before is done with the shared arrays
    if (lane == 31) warp_tokens[warp] = t64, warp_blocks[warp] = b64;
    __syncthreads();
    if (warp == 0) {                            // inclusive sums over the warps
      uint64_t t = warp_tokens[lane], b = warp_blocks[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, t, off), z = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) t += y, b += z;
      }
      warp_tokens[lane] = t;
      warp_blocks[lane] = b;
    }
    __syncthreads();
    const uint64_t tb = warp > 0 ? warp_tokens[warp - 1] : 0, bb = warp > 0 ? warp_blocks[warp - 1] : 0;
    const uint64_t tt = warp_tokens[31], bt = warp_blocks[31];
    const int64_t cu = tokens + (int64_t)(tb + t64) - fresh;
    const int64_t last = blocks + (int64_t)(bb + b64), first = last - max(need, 0);
    const bool fits = need >= 0 && (need == 0 || last <= have) && cu + fresh <= max_new_tokens;
    s_cu[tid] = cu;
    s_len[tid] = len;
    s_first[tid] = (int32_t)min(first, (int64_t)0x7FFFFFFF);
    s_need[tid] = fits ? need : -1;
    if (tid == 0) s_cu[kTableThreads] = tokens + (int64_t)tt;
    if (blockIdx.x == 0) {
      if (r < batch) {
        cu_new[r] = (int32_t)min(cu, (int64_t)0x7FFFFFFF);
        seqlens_out[r] = fits ? len + fresh : len;
        if (r == batch - 1) cu_new[batch] = (int32_t)min(cu + fresh, (int64_t)0x7FFFFFFF);
      }
      const int took = __reduce_add_sync(0xffffffffu, fits ? max(need, 0) : 0);   // at most free_capacity in all
      if (lane == 0 && took > 0) atomicAdd(&s_taken, took);                      // integers: order does not matter
    }
    __syncthreads();
    // table entries: a warp per request, the requests spread over the CTAs
    const int in_chunk = min(batch - r0, kTableThreads);
    for (int q = warp * gridDim.x + blockIdx.x; q < in_chunk; q += 32 * gridDim.x) {
      const int n = s_need[q], at = blocks_of(s_len[q]);
      for (int i = lane; i < n; i += 32)
        block_table[(int64_t)(r0 + q) * max_blocks + at + i] = free_blocks[have - 1 - s_first[q] - i];
    }
    // slots of this CTA's tokens that belong to this chunk's requests
    const int64_t lo = max(i0, s_cu[0]), hi = min(i1, s_cu[kTableThreads]);
    for (int64_t i = lo + tid; i < hi; i += kTableThreads) {
      int a = 0, b = in_chunk - 1;              // the last request that starts at or before token i
      while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (s_cu[mid] <= i) a = mid;
        else b = mid - 1;
      }
      int64_t slot = -1;
      if (s_need[a] >= 0) {
        const int64_t pos = s_len[a] + (i - s_cu[a]);
        const int blk = (int)(pos / 64), old = blocks_of(s_len[a]);
        const int32_t id = blk < old ? block_table[(int64_t)(r0 + a) * max_blocks + blk]
                                     : free_blocks[have - 1 - s_first[a] - (blk - old)];
        slot = (int64_t)id * 64 + pos % 64;
      }
      slots[i] = slot;
    }
    tokens += (int64_t)tt;
    blocks += (int64_t)bt;
  }
  for (int64_t i = max(i0, tokens) + tid; i < i1; i += kTableThreads) slots[i] = -1;   // behind the last token
  if (blockIdx.x == 0) {
    __syncthreads();
    if (tid == 0) num_free_out[0] = (int32_t)(have - s_taken);
    if (tid == 0 && batch == 0) cu_new[0] = 0;
  }
}

}  // namespace smla

extern "C" int smla_extend_block_table(int32_t* block_table, int max_blocks, const int32_t* cache_seqlens,
                                       const int32_t* new_lens, int batch, const int32_t* free_blocks,
                                       int64_t free_capacity, const int32_t* num_free, int64_t max_new_tokens,
                                       int64_t* slot_mapping, int32_t* cu_new, int32_t* seqlens_out,
                                       int32_t* num_free_out, void* stream) {
  if (batch < 0 || max_blocks < 1 || free_capacity < 0 || free_capacity > 0x7FFFFFFF || max_new_tokens < 0 ||
      max_new_tokens > 0x7FFFFFFF)
    return SMLA_ERR_INVALID_ARGUMENT;
  if (!num_free || !cu_new || !num_free_out || (max_new_tokens > 0 && !slot_mapping) ||
      (free_capacity > 0 && !free_blocks))
    return SMLA_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!block_table || !cache_seqlens || !new_lens || !seqlens_out)) return SMLA_ERR_INVALID_ARGUMENT;
  // every CTA reads these while another may already write the results
  if (num_free == num_free_out || (batch > 0 && (cache_seqlens == seqlens_out || new_lens == seqlens_out)))
    return SMLA_ERR_INVALID_ARGUMENT;
  const int64_t want = (max_new_tokens + 2047) / 2048;
  const unsigned ctas = (unsigned)(want < 1 ? 1 : want > 148 ? 148 : want);
  smla::extend_block_table_kernel<<<ctas, smla::kTableThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      block_table, max_blocks, cache_seqlens, new_lens, batch, free_blocks, free_capacity, num_free, max_new_tokens,
      slot_mapping, cu_new, seqlens_out, num_free_out);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SMLA_OK : smla::cuda_failure(e);
}
