// q8_prefill.cu -- grouped-query attention of many new tokens per request over
// the block-scaled 8-bit cache: chunks of prompts and whole prompts.
//
// The formulas are those of q8_decode.cu.  One CTA takes 256 rows of one
// (request, KV head), row = token * group + head of the group, as two tiles of
// 128, and walks the cache blocks (64 keys) that any of its rows sees.
//
// 16 warps:
//   0-3, 4-7  softmax of row tile 0 and 1; thread = row.  A thread reads its
//             row of S from TMEM, writes P (f16) over it and, when its maximum
//             has grown by 2^8, rescales its row of O in TMEM.  Before
//             that the eight warps bring Q in.
//   8-11      producers: codes from global memory to registers (two blocks
//             ahead), to f16, to 128-byte-swizzled shared memory.
//   12, 13    MMA of row tile 0 and 1: S_w = Q_w K^T (both operands in shared
//             memory), then O_w += P_w V (P in TMEM).
// Shared memory: Q 2 x 128 x d, K and V four stages of 64 x d each, f16.
// TMEM: S_0, S_1 double-buffered (4 x 64 columns, P in the first half of each),
// O_0, O_1.  With two buffers S of block i + 1 is there before the softmax of
// block i ends, so a softmax warp waits for no product.
//
// Issuing is what a product costs beside its run time: on this GPU an MMA takes
// its warp about 25 clocks, a commit 85 to 170 and a wait 100, so one warp that
// issued both row tiles' products and told every consumer apart needed 2380
// clocks a block where the tensor cores need 1330.  Hence two issuing warps and
// few commits: S of block i + 2 overwrites P of block i, so it is issued when the
// product of that P is done, and its barrier also says that V of block i and K
// of block i + 2 are read and (to the softmax) that O may be rescaled.
//
// The warps of a row tile may be a block apart, so the barriers between them and
// the products are one per block parity: the one of block i + 2 cannot be reached
// before all four warps are done with block i.
//
// Where the rows do not fill the SMs (a chunk of one request over a long context),
// several CTAs (z) share 256 rows: each takes an equal part of the blocks and leaves a
// normalised fp32 partial, and q8_join_kernel joins them by their lse.  One request, 8
// KV heads, groups of 4, d = 128, alone and shared: 128 tokens on 60000 991 and 133 us, 256
// on 8192 143 and 53, 64 on 8192 141 and 34.
//
// Bound, for 256 rows x 64 keys at d = 128: 1330 clocks of the tensor cores, 1024 of
// the special function units with all exponentials there (a quarter is on the FMA
// pipe).  A step takes 1900 (long loops) to 2300 clocks: the chain of a softmax warp
// from S to P is longer than the products of the other tile.  A CTA takes 8 to 10 us
// beside its steps (finding its request, Q, the output), which is what short prompts
// and documents wait for.  8192 tokens on 8192, 32 heads: 1.5 ms, 1.1 PFLOP/s
// (1.6 ms where the power cap lowers the clocks).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "q8_attention.h"
#include "q8_cache.h"
#include "q8_tma.cuh"
#include "sm100.cuh"

namespace smla {

namespace {

constexpr int kTileRows = 128;            // rows of a tile: the MMA's M
constexpr int kStages = 4;                // cache blocks in shared memory
constexpr int kScaleRing = 8;
constexpr int kThreads = 512;
// Registers of a thread after the split: the warps' shares are what the CTA was
// launched with (512 x 128), which the launch checks.
struct Split {
  static constexpr int kSoftmax = 176, kProducer = 120, kMma = 40;
  static constexpr int kAll = 256 * kSoftmax + 128 * kProducer + 128 * kMma;
  static_assert(kAll <= 65536, "the split must fit what the CTA was launched with");
};
constexpr int kMostSplits = 32;           // CTAs that share 256 rows
// Cache blocks of each, and how many are not shared at all: 64 tokens on 1000 take 20.4 us
// with parts of 4, 22.4 with 6 and 24.3 with 8; on 300 (5 blocks) 19.6 shared, 15.5 not.
constexpr int kLeastBlocks = 4, kAloneBlocks = 8;
constexpr int kWhole = -1, kNothing = -2;
constexpr uint64_t kWaitNs = 2000000000ull;

struct BlockScales {
  float k;                                // key scale; negative where the block is not there
  float rel, unrel;                       // log2 of the value scale over the first one above 0, and 2^-rel
};

template <int D>
struct PrefillShared {                    // at a 1024-byte boundary
  uint8_t q[2][kTileRows * D * 2];
  uint8_t k[kStages][kBlk * D * 2];
  uint8_t v[kStages][kBlk * D * 2];
  BlockScales scales[kScaleRing];
  float2 bias[2 * kTileRows];             // of a row: position, and slope in base 2
  uint64_t full[kStages];                 // K and V of a block
  uint64_t sfull[2][2], pfull[2][2];      // [row tile][block % 2]
  uint64_t odone[2][2], qfull;
  uint32_t tmem;
  int lo, hi;                             // positions that any row sees
  float base;                             // the first value scale above 0, else 0
  Q8Request x;
  int64_t row0, rows_all;
  bool bad;                               // its offsets
  int part;                               // where the result goes: kWhole, kNothing or a partial's slot
};

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

// The phase of `bar` has completed; gives up after kWaitNs.  Inline: a call
// would keep the compiler from moving registers between the warps.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitNs) {
      report_status(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// For a whole warp.  All lanes test the barrier: with lane 0 testing and handing
// its answer on, the kernel took 7 % (d = 128) to 30 % (d = 64) longer.
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const bool ok = bar_wait(bar, parity, status);
  return __all_sync(0xffffffffu, ok);
}

// ---- TMEM: thread i of warp w reads or writes lane 32 (w % 4) + i, 32 columns
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
      "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
      "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]),
      "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]),
      "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}

// kind::f16 with f16 operands and an fp32 accumulator (the fields of
// idesc_bf16_f32 with operand format 0), M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// S = Q K^T over one block: d / 16 MMAs of M = 128, N = 64 issued by one elected
// lane of a converged warp.  A step of 16 along d adds 32 bytes (2 descriptor
// units); the next 64-wide column block is 128 x 128 bytes on in Q (1024) and 64
// x 128 bytes on in K (512).
#define Q8_S_STEP(qo, ko, acc)              \
  "add.u32 la, %1, " qo ";\n\t"             \
  "add.u32 lb, %2, " ko ";\n\t"             \
  "mov.b64 da, {la, %3};\n\t"               \
  "mov.b64 db, {lb, %3};\n\t"               \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " acc ";\n\t"
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint32_t q_lo, uint32_t k_lo, uint32_t hi, uint32_t idesc) {
  if constexpr (D == 128) {
    asm volatile(
        "{\n\t.reg .pred e, pt, pf;\n\t.reg .b32 la, lb;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pt, 1, 0;\n\tsetp.eq.b32 pf, 1, 0;\n\t"
        Q8_S_STEP("0", "0", "pf") Q8_S_STEP("2", "2", "pt") Q8_S_STEP("4", "4", "pt") Q8_S_STEP("6", "6", "pt")
        Q8_S_STEP("1024", "512", "pt") Q8_S_STEP("1026", "514", "pt") Q8_S_STEP("1028", "516", "pt")
        Q8_S_STEP("1030", "518", "pt")
        "}" ::"r"(d_tmem), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, pt, pf;\n\t.reg .b32 la, lb;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pt, 1, 0;\n\tsetp.eq.b32 pf, 1, 0;\n\t"
        Q8_S_STEP("0", "0", "pf") Q8_S_STEP("2", "2", "pt") Q8_S_STEP("4", "4", "pt") Q8_S_STEP("6", "6", "pt")
        "}" ::"r"(d_tmem), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc) : "memory");
  }
}

// O (+)= P V over one block: 4 MMAs of M = 128, N = d, K = 16.  A step is 8
// columns of P in TMEM and 16 rows of 128 bytes of V (128 units).
#define Q8_PV_STEP(ks, acc)                 \
  "add.u32 la, %1, " #ks "*8;\n\t"          \
  "add.u32 lb, %2, " #ks "*128;\n\t"        \
  "mov.b64 db, {lb, %3};\n\t"               \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [la], db, %4, " acc ";\n\t"
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t accumulate_first) {
  asm volatile(
      "{\n\t.reg .pred e, pt, pa;\n\t.reg .b32 la, lb;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pt, 1, 0;\n\tsetp.ne.b32 pa, %5, 0;\n\t"
      Q8_PV_STEP(0, "pa") Q8_PV_STEP(1, "pt") Q8_PV_STEP(2, "pt") Q8_PV_STEP(3, "pt")
      "}" ::"r"(d_tmem), "r"(p_tmem), "r"(v_lo), "r"(hi), "r"(idesc), "r"(accumulate_first)
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The n lowest bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Byte offset of 16-byte chunk `chunk` (8 f16 values) of a row of Q: 64-wide
// column blocks of 128 x 128 bytes, swizzled.
__device__ __forceinline__ uint32_t operand_at(int row, int chunk) {
  return (uint32_t)((chunk >> 3) * (kTileRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

template <int D>
constexpr int kRowLanes = D / 8;          // lanes that read or write a row of q or o

// 2^x for x <= 127 on the FMA pipe (two at a time), for the share of the
// exponentials that the special function units would be waited for: n = round(x)
// by adding 1.5 * 2^23, 2^(x - n) by a degree-4 fit in relative error (2.7e-6 at
// most, 4e-8 in the mean; reweighted least squares on Chebyshev nodes), n added to
// the exponent field (the idea of Schraudolph, "A fast, compact approximation of the
// exponential function", 1999).  Below 2^-126, and for NaN: 2^-126.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 t = add2(x, both(12582912.f));
  const float2 f = fma2(add2(t, both(-12582912.f)), both(-1.f), x);
  float2 r = fma2(both(0.00957009382545948f), f, both(0.05591785907745361f));
  r = fma2(r, f, both(0.240247443318367f));
  r = fma2(r, f, both(0.6931217908859253f));
  r = fma2(r, f, both(0.9999992847442627f));
  r.x = __int_as_float(__float_as_int(r.x) + (__float_as_int(t.x) << 23));
  r.y = __int_as_float(__float_as_int(r.y) + (__float_as_int(t.y) << 23));
  return r;
}

}  // namespace

template <int D, bool kInt8, bool kMods>
__global__ void __launch_bounds__(kThreads, 1) q8_prefill_kernel(const __grid_constant__ Q8Params p,
                                                                  Q8Scratch scratch) {
  constexpr int kStage = kBlk * D * 2;
  extern __shared__ uint8_t raw[];
  PrefillShared<D>& sm = *reinterpret_cast<PrefillShared<D>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y;
  const bool first_cta = blockIdx.x + blockIdx.y + blockIdx.z == 0;
  int32_t* const meta = scratch.meta + 8 * ((size_t)blockIdx.x * p.h_kv + head);
  if (gridDim.z > 1 && blockIdx.z == 0 && tid == 0) meta[0] = 0;

  // ---- which rows: request r may hold the items from cu[r] * group / 256 + r on
  // (one more than its rows fill); the last items, whose tokens see most, first
  const int64_t item = (int64_t)gridDim.x - 1 - blockIdx.x;
  // The owner is the last request whose first item is at or before this one; the
  // thread that tests a request has its lengths ready for the others.
  int r = -1;
  for (int i0 = 0; i0 < p.batch; i0 += kThreads) {
    const int i = i0 + tid;
    bool bad = false, before = false;
    Q8Request mine{0, 0, 0, 0};
    if (i < p.batch) {
      mine = q8_request(p, i, &bad);
      if (bad && first_cta) report_status(p.status, kStatusBadSchedule);
      const int64_t c = p.cu_q ? max(p.cu_q[i], 0) : (int64_t)i * p.s_q;
      before = c * p.group / (2 * kTileRows) + i <= item;
    }
    const int c = __syncthreads_count(before);
    if (c > 0 && r == i0 - 1 && tid == c - 1) {
      sm.x = mine;
      sm.bad = bad;
    }
    if (r == i0 - 1) r += c;
    if (c < kThreads && !first_cta) break;   // the first CTA looks them all over
  }
  if (r < 0) return;
  __syncthreads();
  const Q8Request x = sm.x;
  if (sm.bad) return;
  const int64_t tile = item - ((int64_t)x.q0 * p.group / (2 * kTileRows) + r);
  const int64_t rows_all = (int64_t)x.n * p.group, row0 = tile * 2 * kTileRows;
  if (tile < 0 || row0 >= rows_all) return;
  const bool two = row0 + kTileRows < rows_all;       // the second row tile has rows

  // ---- set-up
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&sm.full[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) {
        bar_init(&sm.sfull[s][b], 1);
        bar_init(&sm.pfull[s][b], 4);
        bar_init(&sm.odone[s][b], 1);
      }
    }
    bar_init(&sm.qfull, 8);
    sm.lo = 0x7FFFFFFF;
    sm.hi = 0;
    sm.row0 = row0;
    sm.rows_all = rows_all;
    sm.part = kWhole;
    mbar_init_fence();
  }
  if (warp == 12) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  const int w = warp >> 2;                            // row tile of a softmax warp
  if (warp < 8) {
    const int64_t row = row0 + tid;                   // of a softmax thread
    int a = 0x7FFFFFFF, b = 0;
    if (row < rows_all) {
      q8_visible(p, x, (int)row / p.group, a, b);
      if (a >= b) a = 0x7FFFFFFF, b = 0;
    }
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    if (lane == 0 && a < b) {
      atomicMin(&sm.lo, a);
      atomicMax(&sm.hi, b);
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int end = (int)min((int64_t)min(sm.hi, 0x7FFFFFFF - 256), (int64_t)p.max_blocks * kBlk);
  int first = sm.lo / kBlk;                           // blocks [first, first + blocks)
  int blocks = sm.lo < end ? (end + kBlk - 1) / kBlk - first : 0;
  if (tid == 0 && sm.hi > (int64_t)p.max_blocks * kBlk) report_status(p.status, kStatusBadBlockTable);

  if (gridDim.z > 1) {                                // the blocks in equal parts over z
    const int least = blocks <= kAloneBlocks ? kAloneBlocks : kLeastBlocks;
    const int per = max((blocks + (int)gridDim.z - 1) / (int)gridDim.z, least);
    const int parts = max((blocks + per - 1) / per, 1), z = blockIdx.z;
    if (tid == 0) {
      sm.part = z >= parts ? kNothing : parts == 1 ? kWhole : ((int)blockIdx.x * p.h_kv + head) * (int)gridDim.z + z;
      if (z == 0 && parts > 1)
        *reinterpret_cast<int4*>(meta) = make_int4(parts, x.q0, (int)row0, (int)rows_all);
    }
    __syncthreads();
    first += z * per;
    blocks = max(min(per, blocks - z * per), 0);
  }
  if (warp < 8) {
    // ================================ softmax ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Split::kSoftmax));
    // This thread's row: token, query head, and which positions it sees.
    int lo = 0, hi = 0x7FFFFFFF;
    int64_t q_at = -1;                                // in q; -1: no row
    // an absent row has no bias either: its scores are 0, and its vote is always the same
    if (kMods && p.slopes) sm.bias[tid] = make_float2(0.f, 0.f);
    if (row0 + tid < rows_all) {
      const int t = (int)(row0 + tid) / p.group, hq = head * p.group + (int)(row0 + tid) - t * p.group;
      q8_visible(p, x, t, lo, hi);
      if (kMods && p.slopes) sm.bias[tid] = make_float2((float)(x.len - x.n + t), p.slopes[hq] * kLog2e);
      q_at = (int64_t)(x.q0 + t) * p.q_token_stride + (int64_t)hq * p.q_head_stride;
    }
    // Q: each row scaled by a power of two, as f16.  A warp copies the 32 rows of its
    // threads into their places as they are, a row by neighbouring lanes, then each
    // thread converts its own row where it lies.
    float row_fac;
    {
      const int sub = lane / kRowLanes<D>, chunk = lane % kRowLanes<D>;
      const uint32_t qs = smem_u32(sm.q[w]);
#pragma unroll 4
      for (int k = 0; k < 32; k += 32 / kRowLanes<D>) {
        const int64_t from = __shfl_sync(0xffffffffu, q_at, k + sub);
        const uint32_t dst = qs + operand_at(32 * (warp & 3) + k + sub, chunk);
        if (from >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p.q + from + 8 * chunk) : "memory");
        else
          sts128(dst, 0, 0, 0, 0);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      auto lo_of = [](uint32_t v) { return __uint_as_float(v << 16); };
      auto hi_of = [](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); };
      const int rr = tid & 127;
      float top = 0.f;
      uint4 u[D / 8];
#pragma unroll
      for (int k = 0; k < D / 8; ++k) u[k] = lds128(qs + operand_at(rr, k));
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const float a = max3(fabsf(lo_of(u[k].x)), fabsf(hi_of(u[k].x)), fabsf(lo_of(u[k].y)));
        const float b = max3(fabsf(hi_of(u[k].y)), fabsf(lo_of(u[k].z)), fabsf(hi_of(u[k].z)));
        top = max3(top, max3(a, b, fabsf(lo_of(u[k].w))), fabsf(hi_of(u[k].w)));
      }
      float up;
      row_pow2(top, up, row_fac);
#pragma unroll
      for (int k = 0; k < D / 8; ++k)
        sts128(qs + operand_at(rr, k), pack_f16(lo_of(u[k].x) * up, hi_of(u[k].x) * up),
               pack_f16(lo_of(u[k].y) * up, hi_of(u[k].y) * up), pack_f16(lo_of(u[k].z) * up, hi_of(u[k].z) * up),
               pack_f16(lo_of(u[k].w) * up, hi_of(u[k].w) * up));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.qfull);
    }
    const uint32_t s_addr = tmem + 128 * w + ((uint32_t)(32 * (warp & 3)) << 16), o_addr = s_addr + 256;
    const float fs = row_fac * p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (w == 0 || two) {
      for (int i = 0; i < blocks; ++i) {
        if (!(ok = bar_wait_warp(&sm.sfull[w][i & 1], (i >> 1) & 1, p.status))) break;
        tc_fence_after();
        const uint32_t sa = s_addr + 64 * (i & 1);
        float S[64];
        tmem_ld32(sa, S);
        tmem_ld32(sa + 32, S + 32);
        // the block's scales come through its (long complete) barrier
        if (!(ok = bar_wait_warp(&sm.full[i % kStages], (i / kStages) & 1, p.status))) break;
        const BlockScales bs = sm.scales[i % kScaleRing];
        const int j0 = (first + i) * kBlk;
        // never 0: a masked score is -inf and has to stay so
        float f = fminf(fmaxf(fs * bs.k, 1e-30f), kMostFactor);
        tmem_wait_ld();
        // capped and biased scores in place (f then is 1)
        if constexpr (kMods) {
          if (p.cap > 0.f) {
            cap_scores<64>(S, f * p.inv_cap_log2, p.cap_log2);
            f = 1.f;
          }
          if (p.slopes) {
            const float2 b = sm.bias[tid];
            const float slope = b.y;
            const float2 d = make_float2(b.x - (float)j0, b.x - (float)(j0 + 1));
#pragma unroll
            for (int j = 0; j < 64; j += 2) {
              const float2 y = mul2(make_float2(S[j], S[j + 1]), both(f));
              S[j] = fmaf(-slope, fabsf(d.x - (float)j), y.x);
              S[j + 1] = fmaf(-slope, fabsf(d.y - (float)j), y.y);
            }
            f = 1.f;
          }
        }
        if (__any_sync(0xffffffffu, j0 < lo || j0 + kBlk > hi) || bs.k < 0.f) {
          const int a = lo - j0, b = bs.k < 0.f ? 0 : hi - j0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {               // columns [a, b) as bits, 32 at a time
            const uint32_t bits = low_bits(b - 32 * q) & ~low_bits(a - 32 * q);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits >> j & 1u)) S[32 * q + j] = -INFINITY;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 64; j += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) top[k] = max3_nan(top[k], S[j + 2 * k], S[j + 2 * k + 1]);
        const float peak = fmaf(max3_nan(top[0], top[1], max3_nan(top[2], top[3], top[3])), f, bs.rel);   // f > 0
        // a NaN score makes the row NaN, and so does an infinite one (inf - inf): by the sum,
        // as ex2_poly keeps neither
        if (!(peak < INFINITY)) l = __int_as_float(0x7FFFFFFF);
        if (__any_sync(0xffffffffu, peak > m + (kHead + kLag))) {
          const float now = fmaxf(m, peak - kHead);
          const float a = now == -INFINITY ? 1.f : ex2(m - now);
          m = now;
          l *= a;
          if (i > 0) {
            // the product of block i - 1 is done when S of block i + 1 is, or the last one
            if (!(ok = i + 1 < blocks ? bar_wait_warp(&sm.sfull[w][(i + 1) & 1], ((i + 1) >> 1) & 1, p.status)
                                      : bar_wait_warp(&sm.odone[w][(i - 1) & 1], ((i - 1) >> 1) & 1, p.status)))
              break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(o_addr + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= a;
              tmem_st32(o_addr + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        const float sub = m == -INFINITY ? 0.f : bs.rel - m;
        float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t P[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = fma2(make_float2(S[32 * c + 2 * j], S[32 * c + 2 * j + 1]), both(f), both(sub));
            if (j % 4 == 3) {
              e = ex2_poly(e);
            } else {
              e.x = ex2(e.x);
              e.y = ex2(e.y);
            }
            sum[j & 1] = add2(sum[j & 1], e);
            P[j] = pack_f16(e.x, e.y);
          }
          tmem_st16(sa + 16 * c, P);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&sm.pfull[w][i & 1]);
        sum[0] = add2(sum[0], sum[1]);
        l = fmaf(sum[0].x + sum[0].y, bs.unrel, l);
      }
      // ---- o = O / l, lse; o goes through Q's place (no product reads it any more),
      // so that whole rows are stored by neighbouring lanes.  What the loop did not
      // need is worked out anew: its registers are S's.
      if (ok && blocks > 0) ok = bar_wait_warp(&sm.odone[w][(blocks - 1) & 1], ((blocks - 1) >> 1) & 1, p.status);
      tc_fence_after();
      if (ok && static_cast<const volatile int&>(sm.part) != kNothing) {
        int me;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(me));
        const volatile PrefillShared<D>& v_sm = sm;
        const int64_t row0 = v_sm.row0, rows_all = v_sm.rows_all;
        const int q0 = v_sm.x.q0, part = v_sm.part, head = blockIdx.y, lane = me & 31, warp = me >> 5;
        const bool none = m == -INFINITY && !(l != l);
        // the scale apart from 1 / l: for values of 2^-100 their product would lose bits
        const float inv = none ? 0.f : 1.f / l, base = v_sm.base;
        const uint32_t qs = smem_u32(sm.q[warp >> 2]);
#pragma unroll 2
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(o_addr + c, o);
          tmem_wait_ld();
          if (part >= 0) {
            float4* dst = reinterpret_cast<float4*>(scratch.o + ((int64_t)part * 2 * kTileRows + me) * D + c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(o[4 * k] * inv * base, o[4 * k + 1] * inv * base, o[4 * k + 2] * inv * base,
                                   o[4 * k + 3] * inv * base);
            continue;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {             // O is not written where there are no blocks
              __nv_bfloat162 b = __floats2bfloat162_rn(none ? 0.f : o[8 * k + 2 * j] * inv * base,
                                                       none ? 0.f : o[8 * k + 2 * j + 1] * inv * base);
              v[j] = *reinterpret_cast<uint32_t*>(&b);
            }
            sts128(qs + operand_at(me & 127, c / 8 + k), v[0], v[1], v[2], v[3]);
          }
        }
        if (part >= 0) {
          scratch.lse[(int64_t)part * 2 * kTileRows + me] = none ? -INFINITY : lse_log2(m, l);
        } else {
          int at = -1;                                  // this thread's row of o and lse
          if (row0 + me < rows_all) {
            const int t = (int)(row0 + me) / p.group;
            at = (q0 + t) * p.h_q + head * p.group + (int)(row0 + me) - t * p.group;
            p.lse[at] = none ? -INFINITY : lse_log2(m, l) * kLn2;
          }
          __syncwarp();
          const int sub = lane / kRowLanes<D>, chunk = lane % kRowLanes<D>;
#pragma unroll 4
          for (int k = 0; k < 32; k += 32 / kRowLanes<D>) {
            const int to = __shfl_sync(0xffffffffu, at, k + sub);
            const uint4 v = lds128(qs + operand_at(32 * (warp & 3) + k + sub, chunk));
            if (to >= 0) reinterpret_cast<uint4*>(p.o + (int64_t)to * D)[chunk] = v;
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ================================ producers ================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split::kProducer));
    // Warp q of 4 converts rows 16q .. 16q + 15 of a block: lane = (row % 8,
    // 16-code chunk % 4); the two rows of a quarter warp land in the even and odd
    // chunks of the swizzle, so the stores have no bank conflicts.
    constexpr int kHalves = D / 64;                   // 64-byte halves of a row of codes
    constexpr int kLoads = 2 * kHalves;               // 16-byte loads of a thread and tile
    const int q = warp - 8, sub = lane >> 2, c4 = lane & 3;
    // Table entries and scales of 32 blocks, one a lane.  The base, the first value scale above
    // 0, is looked for in all 32 or block by block (blocks of zeros before it want none): ragged
    // prompts at d = 128 took 331 us so and 340, at d = 64 153 and 148.
    int page = -1;
    float kscale = -1.f, vscale = 0.f, base_log2 = -INFINITY;
    auto load_entries = [&](int b) {                  // block b: this lane's
      page = -1;
      kscale = -1.f;
      vscale = 0.f;
      if (b < blocks) {
        page = p.block_table[(int64_t)r * p.max_blocks + first + b];
        if (page >= 0 && page < p.num_blocks) {
          kscale = __ldg(p.k_scale + page * p.k_scale_stride + head);
          vscale = __ldg(p.v_scale + page * p.v_scale_stride + head);
        } else {
          report_status(p.status, kStatusBadBlockTable);
          page = -1;
        }
      }
      if constexpr (D == 128)
        if (base_log2 == -INFINITY) {
          const uint32_t above = __ballot_sync(0xffffffffu, vscale > 0.f);
          const float base = __shfl_sync(0xffffffffu, vscale, above ? __ffs(above) - 1 : 0);
          base_log2 = log2f(base);
          if (tid == 256) sm.base = base;
        }
    };
    load_entries(lane);
    const int code_off = (head * kBlk + 16 * q + sub) * D + 16 * c4;
    auto load_tile = [&](uint4 (&codes)[kLoads], int i, const uint8_t* cache, int64_t stride, int pg) {
      // rows behind the request's length count as zero codes
      const int have = x.len - ((first + i) * kBlk + 16 * q + sub);
      const uint8_t* src = cache + pg * stride + code_off;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int part = k / kHalves, half = k % kHalves;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (pg >= 0 && 8 * part < have) v = __ldg(reinterpret_cast<const uint4*>(src + 8 * part * D + 64 * half));
        codes[k] = v;
      }
    };
    // chunks 2 c4 and 2 c4 + 1 (of 8) of row 16 q + sub, whose low three bits are sub's
    const uint32_t at0 = (16 * q + sub) * 128 + (((2 * c4) ^ sub) << 4), at1 = at0 ^ 16u;
    auto store_tile = [&](uint32_t dst, const uint4 (&codes)[kLoads]) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int part = k / kHalves, half = k % kHalves;
        const uint32_t to = dst + half * (kBlk * 128) + 8 * part * 128;
        const uint4 v = codes[k];
        uint32_t f[4];
        Q8Codes<kInt8>::to_f16(v.x, f[0], f[1]);
        Q8Codes<kInt8>::to_f16(v.y, f[2], f[3]);
        sts128(to + at0, f[0], f[1], f[2], f[3]);
        Q8Codes<kInt8>::to_f16(v.z, f[0], f[1]);
        Q8Codes<kInt8>::to_f16(v.w, f[2], f[3]);
        sts128(to + at1, f[0], f[1], f[2], f[3]);
      }
    };
    // This thread's codes of the next two blocks: a load takes longer than a block
    // where many CTAs read the same lines.
    uint4 kc[2][kLoads], vc[2][kLoads];
    float ks[2], vs[2];                               // and their scales
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pg = __shfl_sync(0xffffffffu, page, e);
      ks[e] = __shfl_sync(0xffffffffu, kscale, e);
      vs[e] = __shfl_sync(0xffffffffu, vscale, e);
      if (e < blocks) {
        load_tile(kc[e], e, p.k_cache, p.k_block_bytes, pg);
        load_tile(vc[e], e, p.v_cache, p.v_block_bytes, pg);
      }
    }
    bool ok = true;
    for (int i0 = 0; ok && i0 < blocks; i0 += 2) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = i0 + e;
        if (i >= blocks) break;
        const int st = i % kStages;
        BlockScales bs;
        bs.k = ks[e];
        if constexpr (D == 64)
          if (base_log2 == -INFINITY) {
            base_log2 = log2f(vs[e]);
            if (tid == 256) sm.base = vs[e];
          }
        bs.rel = rel_log2(vs[e], base_log2);
        bs.unrel = ex2(-bs.rel);
        int pg = -1;
        const bool more = i + 2 < blocks;
        if (more) {
          if (((i + 2) & 31) == 0) load_entries(i + 2 + lane);
          pg = __shfl_sync(0xffffffffu, page, (i + 2) & 31);
          ks[e] = __shfl_sync(0xffffffffu, kscale, (i + 2) & 31);
          vs[e] = __shfl_sync(0xffffffffu, vscale, (i + 2) & 31);
        }
        // the stage is free once S of block i - 2 is done, for it stands behind the
        // product of block i - 4; every phase is waited for in turn, as a phase two
        // behind cannot be told from the one asked for
        if (i >= 2) {
          ok = bar_wait_warp(&sm.sfull[0][e], ((i - 2) >> 1) & 1, p.status);
          if (ok && two) ok = bar_wait_warp(&sm.sfull[1][e], ((i - 2) >> 1) & 1, p.status);
          if (!ok) break;
        }
        store_tile(smem_u32(sm.k[st]), kc[e]);
        if (more) load_tile(kc[e], i + 2, p.k_cache, p.k_block_bytes, pg);
        store_tile(smem_u32(sm.v[st]), vc[e]);
        if (more) load_tile(vc[e], i + 2, p.v_cache, p.v_block_bytes, pg);
        if (tid == 256) sm.scales[i % kScaleRing] = bs;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&sm.full[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split::kMma));
    const int ww = warp - 12;                         // row tile
    if (blocks > 0 && (ww == 0 || (ww == 1 && two))) {
      // ================================ MMA ================================
      const uint32_t hi_d = smem_desc_hi_sw128(1024);
      const uint32_t q_lo = smem_desc_lo(smem_u32(sm.q[ww]), 16), k_lo = smem_desc_lo(smem_u32(sm.k[0]), 16);
      const uint32_t v_lo = smem_desc_lo(smem_u32(sm.v[0]), kBlk * 128);   // MN-major: to the next 64 columns
      const uint32_t s_tmem = tmem + 128 * ww, o_tmem = tmem + 256 + 128 * ww;
      constexpr uint32_t kIdS = idesc_f16(kBlk, false), kIdPV = idesc_f16(D, true);
      bool ok = bar_wait_warp(&sm.qfull, 0, p.status);
      // S of block i, into the buffer that P of block i - 2 has left
      auto s_tile = [&](int i) {
        issue_s<D>(s_tmem + 64 * (i & 1), q_lo, k_lo + (uint32_t)(i % kStages) * (kStage >> 4), hi_d, kIdS);
        mma_commit(&sm.sfull[ww][i & 1]);
      };
      for (int i = 0; ok && i < min(2, blocks); ++i) {
        if (!(ok = bar_wait_warp(&sm.full[i], 0, p.status))) break;
        tc_fence_after();
        s_tile(i);
      }
      for (int i = 0; ok && i < blocks; ++i) {
        const int st = i % kStages;
        const bool more = i + 2 < blocks;
        if (more) ok = bar_wait_warp(&sm.full[(i + 2) % kStages], ((i + 2) / kStages) & 1, p.status);
        if (!ok || !(ok = bar_wait_warp(&sm.pfull[ww][i & 1], (i >> 1) & 1, p.status))) break;
        tc_fence_after();
        issue_pv(o_tmem, s_tmem + 64 * (i & 1), v_lo + (uint32_t)st * (kStage >> 4), hi_d, kIdPV, i > 0);
        mma_commit(&sm.odone[ww][i & 1]);
        if (more) {                                   // products of unlike shapes are not ordered by themselves
          if (!(ok = bar_wait_warp(&sm.odone[ww][i & 1], (i >> 1) & 1, p.status))) break;
          s_tile(i + 2);
        }
      }
    }
  }
  // a wait that gave up did so 2 s after the last product was issued: none is in flight
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of CTAs that shared 256 rows: kTeams teams of eight lanes a row, a
// lane's values d = 32 k + 4 (lane % 8) and the next three.  Lane s has the weight of
// part s, and the teams take the parts in turn.  What costs is the trips to L2: one for
// the lse, then one for four parts of each team.  Up to eight parts have one team (512
// tokens on 8192: 91 us, with four teams 94), more have four (64 tokens on 8192, one
// head, 32 parts: 23 us, with one 35).
constexpr int kJoinThreads = 256;
static_assert(kMostSplits <= 32, "a lane for each part");
template <int D, int kTeams>
__global__ void __launch_bounds__(kJoinThreads) q8_join_kernel(const __grid_constant__ Q8Params p, Q8Scratch scratch,
                                                               int splits) {
  constexpr int kLanes = 8 * kTeams;      // of a row
  constexpr int kV = D / 32;
  pdl_wait_primary();
  const int4 ma = *reinterpret_cast<const int4*>(scratch.meta + 8 * (size_t)blockIdx.x);
  const int lane = threadIdx.x % kLanes, in_tile = blockIdx.y * (kJoinThreads / kLanes) + threadIdx.x / kLanes;
  const int parts = ma.x, lane8 = lane & 7, team = lane >> 3;
  const int64_t row = (int64_t)ma.z + in_tile;
  if (parts == 0 || row - threadIdx.x / kLanes >= ma.w) return;   // the CTA's first row
  const int64_t at0 = (int64_t)blockIdx.x * splits * 2 * kTileRows + in_tile;
  const float lse = lane < parts && row < ma.w ? scratch.lse[at0 + (int64_t)lane * 2 * kTileRows] : -INFINITY;
  float top = lse;
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float w = lse == -INFINITY ? 0.f : ex2(lse - top);
  float sum = w;
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  float4 o[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s0 = 0; s0 < parts; s0 += kTeams) {
    const float ws = __shfl_sync(0xffffffffu, w, s0 + team, kLanes);
    if (ws == 0.f) continue;                          // with no weight: what stands there may be no number
    const float4* x = reinterpret_cast<const float4*>(scratch.o + (at0 + (int64_t)(s0 + team) * 2 * kTileRows) * D);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const float4 v = x[8 * k + lane8];
      o[k].x = fmaf(ws, v.x, o[k].x);
      o[k].y = fmaf(ws, v.y, o[k].y);
      o[k].z = fmaf(ws, v.z, o[k].z);
      o[k].w = fmaf(ws, v.w, o[k].w);
    }
  }
  const int t = (int)row / p.group, head = blockIdx.x % p.h_kv, hq = head * p.group + (int)row - t * p.group;
  const int64_t to = (int64_t)(ma.y + t) * p.h_q + hq;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  auto all = [](float v) {                            // over the teams
#pragma unroll
    for (int off = 8; off < kLanes; off *= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    __nv_bfloat162 a = __floats2bfloat162_rn(all(o[k].x) * inv, all(o[k].y) * inv);
    __nv_bfloat162 b = __floats2bfloat162_rn(all(o[k].z) * inv, all(o[k].w) * inv);
    if (team == 0 && row < ma.w)
      reinterpret_cast<uint2*>(p.o + to * D)[8 * k + lane8] =
          make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
  if (lane == 0 && row < ma.w) p.lse[to] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

namespace {

template <int D, bool kInt8, bool kMods>
cudaError_t launch_as(const Q8Params& p, int64_t rows, const Q8Scratch& scratch, int sms, cudaStream_t stream) {
  constexpr int kBytes = sizeof(PrefillShared<D>) + 1024;
  // a register split above what the CTA is launched with would wait for ever
  static std::atomic<int> known{0};
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes at;
    if (const cudaError_t e = cudaFuncGetAttributes(&at, q8_prefill_kernel<D, kInt8, kMods>); e != cudaSuccess)
      return e;
    known.store(regs = at.numRegs, std::memory_order_relaxed);
  }
  if (regs * kThreads < Split::kAll) return cudaErrorInvalidConfiguration;
  static SharedLimit limit;
  if (const cudaError_t e = raise_shared_limit(limit, (const void*)q8_prefill_kernel<D, kInt8, kMods>, kBytes);
      e != cudaSuccess)
    return e;
  const int64_t items = (int64_t)p.total_q * p.group / (2 * kTileRows) + p.batch;
  if (items > 0x7FFFFFFF || p.h_kv > 65535) return cudaErrorInvalidConfiguration;
  // CTAs with rows, as far as the host knows, and how many share one's rows so that
  // they fill the SMs; the workspace has slots for two times the SMs
  const int64_t each = (rows + 2 * kTileRows - 1) / (2 * kTileRows);
  const int64_t busy = std::max<int64_t>(each < items ? std::min(p.batch * each, items) : items, 1) * p.h_kv;
  const int splits =
      (int)std::max<int64_t>(std::min({sms / busy, 2 * sms / (items * p.h_kv), (int64_t)kMostSplits}), 1);
  q8_prefill_kernel<D, kInt8, kMods>
      <<<dim3((unsigned)items, (unsigned)p.h_kv, (unsigned)splits), kThreads, kBytes, stream>>>(p, scratch);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess || splits == 1) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const int teams = splits <= 8 ? 1 : 4;
  cfg.gridDim = dim3((unsigned)(items * p.h_kv), 2 * kTileRows * 8 * teams / kJoinThreads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, teams == 1 ? q8_join_kernel<D, 1> : q8_join_kernel<D, 4>, p, scratch, splits);
}

template <int D, bool kInt8>
cudaError_t launch(const Q8Params& p, int64_t rows, const Q8Scratch& scratch, int sms, cudaStream_t stream) {
  return p.cap > 0.f || p.slopes ? launch_as<D, kInt8, true>(p, rows, scratch, sms, stream)
                                 : launch_as<D, kInt8, false>(p, rows, scratch, sms, stream);
}

}  // namespace

cudaError_t launch_q8_prefill(const Q8Params& p, bool int8, int64_t rows, const Q8Scratch& scratch, int sms,
                              cudaStream_t stream) {
  if (p.d == 128)
    return int8 ? launch<128, true>(p, rows, scratch, sms, stream) : launch<128, false>(p, rows, scratch, sms, stream);
  return int8 ? launch<64, true>(p, rows, scratch, sms, stream) : launch<64, false>(p, rows, scratch, sms, stream);
}

}  // namespace smla
