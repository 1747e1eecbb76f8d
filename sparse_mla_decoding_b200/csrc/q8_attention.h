// q8_attention.h -- launch interface of the attention kernels over the
// block-scaled 8-bit cache (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "q8_cache.h"

namespace smla {

constexpr int kQ8DecodeWarps = 16;       // most warps of a CTA, each with its own range of the work
constexpr int kQ8PartRows = 16;          // rows of a partial
constexpr int64_t kQ8MinVisits = 4;      // least blocks of a CTA's range

// Rows (tokens times the head group) of a request up to which the decode kernel
// runs: it reads the cache once per 16 rows.
constexpr int64_t kQ8DecodeRows = 32;

// Partials of the decode kernel: two slots of kQ8PartRows rows for each warp and for
// each CTA.
struct Q8Scratch {
  float *o, *cta_o;                      // [2 warps or CTAs][kQ8PartRows][d], normalised
  float *lse, *cta_lse;                  // [2 warps or CTAs][kQ8PartRows], log2
  int32_t* meta;                         // [CTAs][8]: the unit that a CTA's range begins inside
};

// `rows`: the most rows (tokens times the head group) of a request, as far as the
// caller knows; it picks the row tile.
cudaError_t launch_q8_decode(const Q8Params& p, bool int8, int rows, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, const Q8Scratch& scratch, int ctas, cudaStream_t stream);

// The tensor-core kernel for many new tokens: no scratch, one CTA per 256 rows.
cudaError_t launch_q8_prefill(const Q8Params& p, bool int8, cudaStream_t stream);

// Raises a kernel's shared memory limit, once per device context (`done`, one per
// kernel, remembers the contexts; after a device reset the context is a new one).
struct SharedLimit {
  std::atomic<void*> done[64];
};
cudaError_t raise_shared_limit(SharedLimit& done, const void* kernel, int bytes);

}  // namespace smla
