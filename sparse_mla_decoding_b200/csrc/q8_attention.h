// q8_attention.h -- launch interface of the attention kernels over the
// block-scaled 8-bit cache (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "q8_cache.h"

namespace smla {

constexpr int kQ8DecodeWarps = 16;       // most warps of a CTA, each with its own range of the work
constexpr int kQ8PartRows = 16;          // rows of a partial
constexpr int64_t kQ8MinVisits = 4;      // least blocks of a CTA's range

// New tokens of a request up to which the decode kernel reads their document bounds
// to leave out blocks that none of them sees.
constexpr int kQ8SpanTokens = 16;

// Which kernel.  Over equally long requests the decode kernel spreads its 16-row tiles
// over all SMs and takes t = tiles / SMs units of time; the tensor-core kernel takes
// waves = ceil(CTAs of 256 rows / SMs) of some 2 units each.  They cross at t between
// 1.8 waves (rows that fill half a CTA) and 2.4.  Measured, decode against tensor
// cores, e4m3, d = 128, 32 heads over 8: 1 request of 60000 tokens, t / waves = 0.22:
// 92 against 764 us, 1.73: 591 against 991; 1 of 8192, 1.73: 95 against 143, 3.46: 174
// against 144; 32 of 4096, 1.73: 101 against 121, 2.6: 142 against 121; d = 64: 8 of
// 4096, 1.73: 44 against 53, 3.46: 74 against 53.
inline bool q8_decode_pays(int64_t batch, int64_t h_kv, int64_t group, int64_t total_q, int64_t max_q, bool docs,
                           int sms) {
  if (max_q > total_q || (docs && max_q > kQ8SpanTokens)) return false;
  const auto tiles = [&](int64_t rows) {              // at most
    return std::min(batch * ((max_q * group + rows - 1) / rows), total_q * group / rows + batch) * h_kv;
  };
  const int64_t waves = (tiles(256) + sms - 1) / sms;
  return 4 * tiles(16) <= 7 * waves * sms;
}

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
