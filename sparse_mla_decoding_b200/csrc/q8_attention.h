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
// Least blocks of a CTA's range: 77 tokens of 8 heads take 10.4 us with 4, 11.5 with 1 and
// 12.4 with 16; 2000 tokens 12.8, 12.5 and 15.6.
constexpr int64_t kQ8MinVisits = 4;

// New tokens of a request up to which the decode kernel reads their document bounds
// to leave out blocks that none of them sees.
constexpr int kQ8SpanTokens = 16;

// Which kernel.  Both spread their work over the SMs; a tile of 16 rows costs the decode
// kernel 0.4 times what 256 rows (or a part of them) cost the tensor-core kernel, whose
// CTAs take some 10 us before and after.  So up to two tiles in place of a CTA go to the
// decode kernel, and so few tiles that they are over before a CTA of the other is.
// Measured, decode against tensor cores, us, 32 heads over 8, d = 128:
//   rows of a request      16          32          48          64         128
//   32 of 4096 tokens   62 / 123   101 / 124   143 / 124   183 / 125
//   4 of 8192           26 / 38     37 / 39     48 / 39     58 / 40     98 / 47
//   1 of 60000          39 / 61     58 / 61     76 / 61     92 / 62    162 / 62
//   1 of 8192           17 / 20     21 / 20     25 / 20     26 / 21     36 / 21
//   1 of 8192, 1 head   15 / 18     15 / 18     15 / 18     15 / 18     17 / 18
inline bool q8_decode_pays(int64_t batch, int64_t h_kv, int64_t group, int64_t total_q, int64_t max_q, bool docs,
                           int sms) {
  if (max_q > total_q || (docs && max_q > kQ8SpanTokens)) return false;
  const auto tiles = [&](int64_t rows) {              // at most, of one head
    return std::min(batch * ((max_q * group + rows - 1) / rows), total_q * group / rows + batch);
  };
  return tiles(16) <= 2 * tiles(256) || 16 * tiles(16) * h_kv <= sms;
}

// Partials of the decode kernel: two slots of kQ8PartRows rows for each warp and for
// each CTA.  The tensor-core kernel has its slots of 256 rows in `o` and `lse` (two for
// each SM) and one entry of `meta` for each 256 rows that several CTAs share.
struct Q8Scratch {
  float *o, *cta_o;                      // [2 warps or CTAs][kQ8PartRows][d], normalised
  float *lse, *cta_lse;                  // [2 warps or CTAs][kQ8PartRows], log2
  int32_t* meta;                         // [CTAs][8]: the unit that a CTA's range begins inside
};

// `rows`: the most rows (tokens times the head group) of a request, as far as the
// caller knows; it picks the row tile.
cudaError_t launch_q8_decode(const Q8Params& p, bool int8, int rows, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, const Q8Scratch& scratch, int ctas, cudaStream_t stream);

// The tensor-core kernel for many new tokens, one CTA per 256 rows or, where these would
// not fill the SMs, several; `rows` as above.
cudaError_t launch_q8_prefill(const Q8Params& p, bool int8, int64_t rows, const Q8Scratch& scratch, int sms,
                              cudaStream_t stream);

// Raises a kernel's shared memory limit, once per device context (`done`, one per
// kernel, remembers the contexts; after a device reset the context is a new one).
struct SharedLimit {
  std::atomic<void*> done[64];
};
cudaError_t raise_shared_limit(SharedLimit& done, const void* kernel, int bytes);

}  // namespace smla
