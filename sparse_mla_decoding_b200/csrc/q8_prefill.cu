// q8_prefill.cu -- grouped-query attention of many new tokens per request over
// the block-scaled 8-bit cache: chunks of prompts and whole prompts.
//
// The formulas are those of q8_decode.cu.  One CTA takes 256 rows of one
// (request, KV head), row = token * group + head of the group, as two tiles of
// 128, and walks the key tiles of 128 positions (two cache blocks) that any of
// its rows sees.  Bound by the tensor cores: 4 * 256 * 128 * d flop a key tile,
// 2048 clocks at d = 128 and the full M = 128 rate; a tile also takes 32768
// exponentials, 2048 clocks of the SM's special function units.
//
// 16 warps:
//   0-3, 4-7  softmax of row tile 0 and 1; thread = row.  A thread reads its
//             row of S from TMEM, writes P (f16) over it and, when its maximum
//             grows by more than 2^8, rescales its row of O in TMEM.
//   8-11      producers: codes from global memory to registers (one tile
//             ahead), to f16, to 128-byte-swizzled shared memory.
//   12        MMA: S_w = Q_w K^T (both operands in shared memory), then
//             O_w += P_w V (P in TMEM), the two row tiles in turn, so one
//             tile's products run under the other's softmax.
// Shared memory: Q 2 x 128 x d, K and V two stages of 128 x d each, f16.
// TMEM: S_0, S_1 (128 columns each, P in the first half), O_0, O_1.
// Registers are moved from the eight other warps to the softmax warps.
#include <cuda_runtime.h>

#include <cstdint>

#include "q8_attention.h"
#include "q8_cache.h"
#include "q8_tma.cuh"
#include "sm100.cuh"

namespace smla {

namespace {

constexpr int kTileRows = 128;            // rows of a tile: the MMA's M
constexpr int kTileKeys = 128;            // positions of a key tile
constexpr int kThreads = 512;
// Registers of a thread after the split: the warps' shares are what the CTA was
// launched with (512 x 128), which the launch checks.
constexpr int kSoftmaxRegs = 192, kProducerRegs = 72, kMmaRegs = 56;
constexpr int kSplitRegs = 256 * kSoftmaxRegs + 128 * kProducerRegs + 128 * kMmaRegs;
static_assert(kSplitRegs <= 65536, "the split must fit what the CTA was launched with");
constexpr uint64_t kWaitNs = 2000000000ull;

struct KeyScales {                        // of the two cache blocks of a key tile
  float k[2];                             // key scale; 0 where the block is not there
  float rel[2], unrel[2];                 // log2 of the value scale over the first one's, and 2^-rel
  uint32_t there;                         // bit per block
};

template <int D>
struct PrefillShared {                    // at a 1024-byte boundary
  uint8_t q[2][kTileRows * D * 2];
  uint8_t k[2][kTileKeys * D * 2];
  uint8_t v[2][kTileKeys * D * 2];
  KeyScales scales[4];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2];
  uint32_t tmem;
  int lo, hi;                             // positions that any row sees
  float base_log2;
  int q0, r, blocks;
  int64_t row0, rows_all;
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}
// kind::f16 with f16 operands and an fp32 accumulator (the fields of
// idesc_bf16_f32 with operand format 0), M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// S = Q K^T for d = 64 or 128: d / 16 MMAs of M = 128, N = 128 issued by one
// elected lane of a converged warp.  A step of 16 along d adds 32 bytes (2
// descriptor units), a 64-wide column block 128 rows x 128 bytes (1024).
#define Q8_S_STEP(off, acc)                 \
  "add.u32 la, %1, " off ";\n\t"            \
  "add.u32 lb, %2, " off ";\n\t"            \
  "mov.b64 da, {la, %3};\n\t"               \
  "mov.b64 db, {lb, %3};\n\t"               \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " acc ";\n\t"
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint32_t q_lo, uint32_t k_lo, uint32_t hi, uint32_t idesc) {
  if constexpr (D == 128) {
    asm volatile(
        "{\n\t.reg .pred e, pt, pf;\n\t.reg .b32 la, lb;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pt, 1, 0;\n\tsetp.eq.b32 pf, 1, 0;\n\t"
        Q8_S_STEP("0", "pf") Q8_S_STEP("2", "pt") Q8_S_STEP("4", "pt") Q8_S_STEP("6", "pt")
        Q8_S_STEP("1024", "pt") Q8_S_STEP("1026", "pt") Q8_S_STEP("1028", "pt") Q8_S_STEP("1030", "pt")
        "}" ::"r"(d_tmem), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc) : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, pt, pf;\n\t.reg .b32 la, lb;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pt, 1, 0;\n\tsetp.eq.b32 pf, 1, 0;\n\t"
        Q8_S_STEP("0", "pf") Q8_S_STEP("2", "pt") Q8_S_STEP("4", "pt") Q8_S_STEP("6", "pt")
        "}" ::"r"(d_tmem), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc) : "memory");
  }
}

// O (+)= P V over 128 keys: 8 MMAs of M = 128, N = d, K = 16.  A step is 8
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
      Q8_PV_STEP(4, "pt") Q8_PV_STEP(5, "pt") Q8_PV_STEP(6, "pt") Q8_PV_STEP(7, "pt")
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

// Byte offset of 16-byte chunk `chunk` (8 f16 values) of a row in an operand
// tile of 128 rows: 64-wide column blocks of 128 x 128 bytes, swizzled.
__device__ __forceinline__ uint32_t operand_at(int row, int chunk) {
  return (uint32_t)((chunk >> 3) * (kTileRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

}  // namespace

template <int D, bool kInt8, bool kMods>
__global__ void __launch_bounds__(kThreads, 1) q8_prefill_kernel(const __grid_constant__ Q8Params p) {
  constexpr int kStage = kTileKeys * D * 2;
  extern __shared__ uint8_t raw[];
  PrefillShared<D>& sm = *reinterpret_cast<PrefillShared<D>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y;

  // ---- which rows: request r may hold the items from cu[r] * group / 256 + r on
  // (one more than its rows fill); the last items, whose tokens see most, first
  const int64_t item = (int64_t)gridDim.x - 1 - blockIdx.x;
  int r = -1;
  for (int i0 = 0; i0 < p.batch; i0 += kThreads) {
    const int i = i0 + tid;
    bool before = false;
    if (i < p.batch) {
      const int64_t c = p.cu_q ? max(p.cu_q[i], 0) : (int64_t)i * p.s_q;
      before = c * p.group / (2 * kTileRows) + i <= item;
    }
    const int c = __syncthreads_count(before);
    r += c;
    if (c < kThreads) break;
  }
  if (r < 0) return;
  bool bad;
  const Q8Request x = q8_request(p, r, &bad);
  if (bad) {
    if (tid == 0) report_status(p.status, kStatusBadSchedule);
    return;
  }
  const int64_t tile = item - ((int64_t)x.q0 * p.group / (2 * kTileRows) + r);
  const int64_t rows_all = (int64_t)x.n * p.group, row0 = tile * 2 * kTileRows;
  if (tile < 0 || row0 >= rows_all) return;
  const bool two = row0 + kTileRows < rows_all;       // the second row tile has rows

  // ---- set-up
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      bar_init(&sm.kfull[s], 4);
      bar_init(&sm.vfull[s], 4);
      bar_init(&sm.kempty[s], 1);
      bar_init(&sm.vempty[s], 1);
      bar_init(&sm.sfull[s], 2);
      bar_init(&sm.pfull[s], 4);
      bar_init(&sm.ofull[s], 1);
    }
    sm.lo = 0x7FFFFFFF;
    sm.hi = 0;
    sm.q0 = x.q0;
    sm.r = r;
    sm.row0 = row0;
    sm.rows_all = rows_all;
    mbar_init_fence();
  }
  if (warp == 12) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  const int w = warp >> 2;                            // row tile of a softmax warp
  const int64_t row = row0 + tid;                     // of a softmax thread
  const int t = (int)(row / p.group), hq = head * p.group + (int)(row % p.group);
  const bool live = warp < 8 && row < rows_all;
  int lo = 0, hi = 0x7FFFFFFF;
  float row_fac = 1.f;
  if (warp < 8) {
    int a = 0x7FFFFFFF, b = 0;
    if (live) {
      q8_visible(p, x, t, lo, hi);
      if (lo < hi) a = lo, b = hi;
    }
    a = __reduce_min_sync(0xffffffffu, a);
    b = __reduce_max_sync(0xffffffffu, b);
    if (lane == 0 && a < b) {
      atomicMin(&sm.lo, a);
      atomicMax(&sm.hi, b);
    }
    // Q: this row, scaled by a power of two, as f16 (read twice, the second time from cache)
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(x.q0 + (live ? t : 0)) * p.q_token_stride +
                                                      (int64_t)hq * p.q_head_stride);
    float top = 0.f;
    auto lo_of = [](uint32_t v) { return __uint_as_float(v << 16); };
    auto hi_of = [](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); };
#pragma unroll 4
    for (int k = 0; k < D / 8; ++k) {
      const uint4 u = live ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(lo_of(v[j])), fabsf(hi_of(v[j]))));
    }
    float up, down;
    row_pow2(top, up, down);
    row_fac = down;
    const uint32_t qs = smem_u32(sm.q[w]);
#pragma unroll 4
    for (int k = 0; k < D / 8; ++k) {
      const uint4 u = live ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
      uint32_t f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = pack_f16(lo_of(v[j]) * up, hi_of(v[j]) * up);
      sts128(qs + operand_at(tid & 127, k), f[0], f[1], f[2], f[3]);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int end = (int)min((int64_t)min(sm.hi, 0x7FFFFFFF - 256), (int64_t)p.max_blocks * kBlk);
  const int first = sm.lo / kTileKeys;                // key tiles [first, last)
  const int last = sm.lo < end ? (end + kTileKeys - 1) / kTileKeys : first;
  if (tid == 0 && sm.hi > (int64_t)p.max_blocks * kBlk) report_status(p.status, kStatusBadBlockTable);
  const int tiles = max(last - first, 0);
  if (tid == 256) sm.blocks = (end + kBlk - 1) / kBlk;

  if (warp < 8) {
    // ================================ softmax ================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const uint32_t s_addr = tmem + 128 * w + ((uint32_t)(32 * (warp & 3)) << 16), o_addr = s_addr + 256;
    const float slope = live && p.slopes ? p.slopes[hq] * kLog2e : 0.f;
    const float pos = (float)(x.len - x.n + t);
    const float fs = row_fac * p.scale * kLog2e;
    const float fc = p.cap > 0.f ? row_fac * p.scale / p.cap : 0.f, cl = p.cap * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (w == 0 || two) {
      for (int i = 0; i < tiles; ++i) {
        if (!(ok = bar_wait_warp(&sm.sfull[w], i & 1, p.status))) break;
        tc_fence_after();
        const volatile KeyScales& ks = sm.scales[i & 3];   // read where used: S needs the registers
        float S[128];
        tmem_ld32(s_addr, S);
        tmem_ld32(s_addr + 32, S + 32);
        tmem_ld32(s_addr + 64, S + 64);
        tmem_ld32(s_addr + 96, S + 96);
        tmem_wait_ld();
        const int j0 = (first + i) * kTileKeys;
        // never 0: a masked score is -inf and has to stay so
        float f[2] = {fmaxf(fs * ks.k[0], 1e-30f), fmaxf(fs * ks.k[1], 1e-30f)};
        // capped and biased scores in place (f then is 1)
        if constexpr (kMods) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (p.cap > 0.f) {
              cap_scores<32>(S + 64 * h, fc * ks.k[h], cl);
              cap_scores<32>(S + 64 * h + 32, fc * ks.k[h], cl);
              f[h] = 1.f;
            }
            if (p.slopes) {
              float2 d = make_float2(pos - (float)(j0 + 64 * h), pos - (float)(j0 + 64 * h + 1));
#pragma unroll
              for (int j = 0; j < 64; j += 2) {
                const float2 x = mul2(make_float2(S[64 * h + j], S[64 * h + j + 1]), both(f[h]));
                S[64 * h + j] = fmaf(-slope, fabsf(d.x - (float)j), x.x);
                S[64 * h + j + 1] = fmaf(-slope, fabsf(d.y - (float)j), x.y);
              }
              f[h] = 1.f;
            }
          }
        }
        if (__any_sync(0xffffffffu, j0 < lo || j0 + kTileKeys > hi) || ks.there != 3u) {
          int a = lo - j0, b = hi - j0;
          if (!(ks.there & 1u)) a = max(a, kBlk);
          if (!(ks.there & 2u)) b = min(b, kBlk);
#pragma unroll
          for (int q = 0; q < 4; ++q) {               // columns [a, b) as bits, 32 at a time
            const uint32_t bits = low_bits(b - 32 * q) & ~low_bits(a - 32 * q);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(bits >> j & 1u)) S[32 * q + j] = -INFINITY;
          }
        }
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 64; j += 4) {
            a[0] = max3(a[0], S[64 * h + j], S[64 * h + j + 1]);
            a[1] = max3(a[1], S[64 * h + j + 2], S[64 * h + j + 3]);
          }
          top[h] = fmaxf(a[0], a[1]);
          top[h] = fmaf(top[h], f[h], ks.rel[h]);      // f > 0
        }
        const float peak = fmaxf(top[0], top[1]);
        if (__any_sync(0xffffffffu, peak > m + 8.f)) {
          const float now = fmaxf(m, peak);
          const float a = now == -INFINITY ? 1.f : ex2(m - now);
          m = now;
          l *= a;
          if (i > 0) {                                // S of this tile complete: so is every product before it
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(o_addr + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= a;
              tmem_st16(o_addr + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sub = m == -INFINITY ? 0.f : ks.rel[h] - m;
          float2 sum = both(0.f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t P[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int at = 64 * h + 32 * c + 2 * j;
              float2 e = fma2(make_float2(S[at], S[at + 1]), both(f[h]), both(sub));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum = add2(sum, e);
              P[j] = pack_f16(e.x, e.y);
            }
            tmem_st16(s_addr + 32 * h + 16 * c, P);
          }
          l = fmaf(sum.x + sum.y, ks.unrel[h], l);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&sm.pfull[w]);
      }
      // ---- o = O / l, lse; what the loop did not need is taken from shared memory again
      if (ok && tiles > 0) ok = bar_wait_warp(&sm.ofull[w], 0, p.status);
      tc_fence_after();
      if (ok) {
        int me;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(me));
        const int64_t row = *(volatile int64_t*)&sm.row0 + me;
        const bool live = row < *(volatile int64_t*)&sm.rows_all;
        const int64_t at = (*(volatile int*)&sm.q0 + row / p.group) * p.h_q + blockIdx.y * p.group + row % p.group;
        const bool none = l == 0.f;
        const float inv = none ? 0.f : ex2(sm.base_log2) / l;
        if (live) p.lse[at] = none ? -INFINITY : (m + log2f(l)) * kLn2;
        __nv_bfloat16* dst = p.o + at * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(o_addr + c, o);
          tmem_wait_ld();
          uint32_t v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {               // O is not written where there are no tiles
            __nv_bfloat162 b = __floats2bfloat162_rn(none ? 0.f : o[2 * j] * inv, none ? 0.f : o[2 * j + 1] * inv);
            v[j] = *reinterpret_cast<uint32_t*>(&b);
          }
          if (live) {
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp < 12) {
    // ================================ producers ================================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // Warp q of 4 converts rows 16q .. 16q + 15 of each cache block: lane = (row
    // % 8, 16-code chunk % 4); the two rows of a quarter warp land in the even
    // and odd chunks of the swizzle, so the stores have no bank conflicts.
    constexpr int kHalves = D / 64;                   // 64-byte halves of a row of codes
    constexpr int kLoads = 2 * 2 * kHalves;           // 16-byte loads of a thread and key tile
    const int q = warp - 8, sub = lane >> 2, c4 = lane & 3;
    asm volatile("bar.sync 1, 128;" ::: "memory");    // sm.blocks
    // Table entries and scales of 32 blocks (16 key tiles), one a lane.
    int page = -1;
    float kscale = 0.f, vscale = 0.f;
    auto load_entries = [&](int b) {
      page = -1;
      kscale = vscale = 0.f;
      const volatile PrefillShared<D>& again = sm;    // seldom used, so not kept in registers
      if (b >= again.lo / kBlk && b < again.blocks) { // a block that some row sees
        page = p.block_table[(int64_t)again.r * p.max_blocks + b];
        if (page >= 0 && page < p.num_blocks) {
          kscale = __ldg(p.k_scale + page * p.k_scale_stride + head);
          vscale = __ldg(p.v_scale + page * p.v_scale_stride + head);
        } else {
          report_status(p.status, kStatusBadBlockTable);
          page = -1;
        }
      }
    };
    load_entries(2 * first + lane);
    const float v0 = __shfl_sync(0xffffffffu, vscale, 0);
    if (tid == 256) sm.base_log2 = v0 > 0.f ? log2f(v0) : 0.f;
    uint4 raw_codes[kLoads];                          // this thread's codes of one tile, keys or values
    const int code_off = (head * kBlk + 16 * q + sub) * D + 16 * c4;
    auto load_tile = [&](int i, const uint8_t* cache, int64_t stride, int pg0, int pg1) {
      // rows behind the request's length count as zero codes
      const int have = x.len - ((first + i) * kTileKeys + 16 * q + sub);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int pg = b ? pg1 : pg0;
        const uint8_t* src = cache + pg * stride + code_off;
#pragma unroll
        for (int k = 0; k < kLoads / 2; ++k) {
          const int part = k / kHalves, half = k % kHalves;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (pg >= 0 && b * kBlk + 8 * part < have)
            v = __ldg(reinterpret_cast<const uint4*>(src + 8 * part * D + 64 * half));
          raw_codes[b * (kLoads / 2) + k] = v;
        }
      }
    };
    // chunks 2 c4 and 2 c4 + 1 (of 8) of row 16 q + sub, whose low three bits are sub's
    const uint32_t at0 = (16 * q + sub) * 128 + (((2 * c4) ^ sub) << 4), at1 = at0 ^ 16u;
    auto store_tile = [&](uint32_t dst) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int b = k / (2 * kHalves), part = (k / kHalves) & 1, half = k % kHalves;
        const uint32_t to = dst + half * (kTileKeys * 128) + (kBlk * b + 8 * part) * 128;
        const uint4 v = raw_codes[k];
        uint32_t f[4];
        Q8Codes<kInt8>::to_f16(v.x, f[0], f[1]);
        Q8Codes<kInt8>::to_f16(v.y, f[2], f[3]);
        sts128(to + at0, f[0], f[1], f[2], f[3]);
        Q8Codes<kInt8>::to_f16(v.z, f[0], f[1]);
        Q8Codes<kInt8>::to_f16(v.w, f[2], f[3]);
        sts128(to + at1, f[0], f[1], f[2], f[3]);
      }
    };
    int pg0 = __shfl_sync(0xffffffffu, page, 0), pg1 = __shfl_sync(0xffffffffu, page, 1);
    if (tiles > 0) load_tile(0, p.k_cache, p.k_block_bytes, pg0, pg1);
    bool ok = true;
    for (int i = 0; i < tiles; ++i) {
      const int st = i & 1, at = 2 * (i & 15);
      const uint32_t parity = ((i >> 1) & 1) ^ 1;
      // keys
      if (!(ok = bar_wait_warp(&sm.kempty[st], parity, p.status))) break;
      store_tile(smem_u32(sm.k[st]));
      load_tile(i, p.v_cache, p.v_block_bytes, pg0, pg1);                      // the values come in while the keys go out
      const float k0 = __shfl_sync(0xffffffffu, kscale, at), k1 = __shfl_sync(0xffffffffu, kscale, at + 1);
      const float w0 = __shfl_sync(0xffffffffu, vscale, at), w1 = __shfl_sync(0xffffffffu, vscale, at + 1);
      if (tid == 256) {
        KeyScales ks;
        ks.k[0] = k0, ks.k[1] = k1;
        const float from = sm.base_log2;
        ks.rel[0] = rel_log2(w0, from), ks.rel[1] = rel_log2(w1, from);
        ks.unrel[0] = ex2(-ks.rel[0]), ks.unrel[1] = ex2(-ks.rel[1]);
        ks.there = (pg0 >= 0 ? 1u : 0u) | (pg1 >= 0 ? 2u : 0u);
        sm.scales[i & 3] = ks;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.kfull[st]);
      // values
      if (!(ok = bar_wait_warp(&sm.vempty[st], parity, p.status))) break;
      store_tile(smem_u32(sm.v[st]));
      if (i + 1 < tiles) {
        if ((i & 15) == 15) load_entries(2 * (first + i + 1) + lane);
        const int nx = 2 * ((i + 1) & 15);
        pg0 = __shfl_sync(0xffffffffu, page, nx);
        pg1 = __shfl_sync(0xffffffffu, page, nx + 1);
        load_tile(i + 1, p.k_cache, p.k_block_bytes, pg0, pg1);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&sm.vfull[st]);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == 12 && tiles > 0) {
      // ================================ MMA ================================
      const uint32_t hi_d = smem_desc_hi_sw128(1024);
      const uint32_t q_lo[2] = {smem_desc_lo(smem_u32(sm.q[0]), 16), smem_desc_lo(smem_u32(sm.q[1]), 16)};
      const uint32_t k_lo = smem_desc_lo(smem_u32(sm.k[0]), 16);
      const uint32_t v_lo = smem_desc_lo(smem_u32(sm.v[0]), kTileKeys * 128);   // MN-major: to the next 64 columns
      constexpr uint32_t kIdS = idesc_f16(kTileKeys, false), kIdPV = idesc_f16(D, true);
      auto s_tile = [&](int i, int ww) {
        issue_s<D>(tmem + 128 * ww, q_lo[ww], k_lo + (uint32_t)(i & 1) * (kStage >> 4), hi_d, kIdS);
        mma_commit(&sm.sfull[ww]);
        // the scales beside the tile come through this thread's wait on kfull
        if (lane == 0) mbar_arrive1(&sm.sfull[ww]);
      };
      bool ok = bar_wait_warp(&sm.kfull[0], 0, p.status);
      if (ok) {
        tc_fence_after();
        s_tile(0, 0);
        if (two) s_tile(0, 1);
        mma_commit(&sm.kempty[0]);
      }
      for (int i = 0; ok && i < tiles; ++i) {
        const int st = i & 1;
        ok = bar_wait_warp(&sm.vfull[st], (i >> 1) & 1, p.status);
        const bool more = i + 1 < tiles;
        if (ok && more) ok = bar_wait_warp(&sm.kfull[st ^ 1], ((i + 1) >> 1) & 1, p.status);
        for (int ww = 0; ok && ww < (two ? 2 : 1); ++ww) {
          if (!(ok = bar_wait_warp(&sm.pfull[ww], i & 1, p.status))) break;
          tc_fence_after();
          issue_pv(tmem + 256 + 128 * ww, tmem + 128 * ww, v_lo + (uint32_t)st * (kStage >> 4), hi_d, kIdPV, i > 0);
          if (more) s_tile(i + 1, ww);
          else mma_commit(&sm.ofull[ww]);
        }
        if (ok) {
          mma_commit(&sm.vempty[st]);
          if (more) mma_commit(&sm.kempty[st ^ 1]);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

template <int D, bool kInt8, bool kMods>
cudaError_t launch_as(const Q8Params& p, cudaStream_t stream) {
  constexpr int kBytes = sizeof(PrefillShared<D>) + 1024;
  cudaFuncAttributes at;
  if (const cudaError_t e = cudaFuncGetAttributes(&at, q8_prefill_kernel<D, kInt8, kMods>); e != cudaSuccess) return e;
  // a register split above what the CTA is launched with would wait for ever
  if (at.numRegs * kThreads < kSplitRegs) return cudaErrorInvalidConfiguration;
  if (const cudaError_t e = cudaFuncSetAttribute(q8_prefill_kernel<D, kInt8, kMods>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
      e != cudaSuccess)
    return e;
  const int64_t items = (int64_t)p.total_q * p.group / (2 * kTileRows) + p.batch;
  if (items > 0x7FFFFFFF || p.h_kv > 65535) return cudaErrorInvalidConfiguration;
  q8_prefill_kernel<D, kInt8, kMods><<<dim3((unsigned)items, (unsigned)p.h_kv), kThreads, kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool kInt8>
cudaError_t launch(const Q8Params& p, cudaStream_t stream) {
  return p.cap > 0.f || p.slopes ? launch_as<D, kInt8, true>(p, stream) : launch_as<D, kInt8, false>(p, stream);
}

}  // namespace

cudaError_t launch_q8_prefill(const Q8Params& p, bool int8, cudaStream_t stream) {
  if (p.d == 128) return int8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return int8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace smla
