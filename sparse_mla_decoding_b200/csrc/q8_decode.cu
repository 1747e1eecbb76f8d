// q8_decode.cu -- grouped-query attention of a few new tokens per request over
// the block-scaled 8-bit cache.
//
// For new token t of a request (position p = len - n + t) and query head h of
// KV head h / group, over the visible cache positions j:
//   x_j = scale <q, k_j>;  x_j = cap tanh(x_j / cap) with a cap;
//   x_j -= slope_h |p - j| with slopes;
//   lse = ln sum_j exp(x_j),  o = sum_j exp(x_j - lse) v_j.
//
// Work: one visit is one cache block of one (request, row tile, KV head); the rows
// of a tile are (token, head of the group) pairs, so a block's codes are read once
// for the whole group.  All visits, in (request, row tile, head, block) order, are
// cut into equal ranges, one per warp; a warp walks its range alone, with its own
// ring of TMA tiles, and no warp waits for another.  A range that holds a whole
// (request, tile, head) writes o itself; pieces of one go to the workspace as
// normalised partials that q8_combine_kernel merges by their lse.
//
// Products: S^T = K Q^T and O^T = V^T P^T on m16n8k16, so the cache's codes fill
// the 16-row side and a tile has 8 rows (one MMA column block) or 16 (two): a group
// of 8 heads wastes nothing, where rows on the 16-row side would double the
// products and the softmax.  The codes go to f16 in registers, once for all rows.
//
// Numbers: codes are exact in f16 and q is scaled by a power of two per row, so S
// has no input rounding and the scales multiply in fp32.  A value scale rides in
// the exponent,
//   p_j = 2^(x_j + log2 v_scale - m),
// so one accumulator holds blocks of different scales; the sum of the softmax
// takes the factor out again per block.  P is rounded to f16 once (2^-11).
//
// Bound by HBM: d + 1/16 bytes a key, value and head; what has to keep up is the
// conversion, about 470 instructions a warp and block (16 KB at d = 128).
#include <cuda_runtime.h>

#include <cstdint>

#include "q8_attention.h"
#include "q8_cache.h"
#include "q8_tma.cuh"
#include "sm100.cuh"

namespace smla {

namespace {

constexpr int kPartRows = kQ8PartRows;    // rows of a partial slot
constexpr int kRing = 64;                 // visits whose table entries a warp keeps
constexpr int kSpanTokens = 16;           // document bounds are scanned up to this many new tokens
constexpr uint64_t kWaitNs = 2000000000ull;

// Warps of a CTA and tiles of a warp's ring: 192 KB of tiles in all.  8 rows take
// under 170 registers, 16 rows up to 255.
template <int NT>
constexpr int kWarpsOf = NT == 1 ? 12 : 8;
template <int D, int NT>
constexpr int kTileSlots = 192 * 1024 / (kBlk * D * kWarpsOf<NT>);

struct Entry {                            // one visit of the ring
  int block, head;                        // cache block (-1: nothing to read) and KV head
  float k_scale, v_scale;
};

// Blocks [first, first + count) that any row of the request sees; at least one,
// so that every request with new tokens gets its outputs written.
__device__ __forceinline__ void block_span(const Q8Params& p, const Q8Request& x, int& first, int& count) {
  int lo = 0, hi = x.len;
  if (p.docs && x.n <= kSpanTokens) {
    lo = x.len;
    hi = 0;
    for (int t = 0; t < x.n; ++t) {
      int a, b;
      q8_visible(p, x, t, a, b);
      if (a < b) {
        lo = min(lo, a);
        hi = max(hi, b);
      }
    }
  }
  const int end = min((hi + kBlk - 1) / kBlk, p.max_blocks);
  first = min(lo / kBlk, p.max_blocks - 1);
  count = max(1, end - first);
}

template <int NT>
__device__ __forceinline__ int row_tiles(const Q8Params& p, int n) {
  return (n * p.group + 8 * NT - 1) / (8 * NT);
}

template <int NT>
__device__ __forceinline__ int64_t visits_of(const Q8Params& p, int r) {
  bool bad;
  const Q8Request x = q8_request(p, r, &bad);
  if (x.n == 0) return 0;
  int first, count;
  block_span(p, x, first, count);
  return (int64_t)p.h_kv * row_tiles<NT>(p, x.n) * count;
}

// A position in the list of visits.
template <int NT>
struct Cursor {
  int r;
  Q8Request x;
  int first, count, units, unit, blk;

  __device__ __forceinline__ void load(const Q8Params& p) {
    bool bad;
    x = q8_request(p, r, &bad);
    block_span(p, x, first, count);
    units = p.h_kv * row_tiles<NT>(p, x.n);
  }
  // to visit `off` of the requests from r on
  __device__ __forceinline__ void seek(const Q8Params& p, int64_t off) {
    while (true) {
      load(p);
      const int64_t have = (int64_t)units * count;
      if (off < have) break;
      off -= have;
      ++r;
    }
    unit = (int)(off / count);
    blk = (int)(off % count);
  }
  __device__ __forceinline__ void next_request(const Q8Params& p) {
    do {
      ++r;
      if (r >= p.batch) return;
      load(p);
    } while (units == 0);
    unit = blk = 0;
  }
  __device__ __forceinline__ void step(const Q8Params& p) {
    if (++blk < count) return;
    blk = 0;
    if (++unit < units) return;
    next_request(p);
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 f16 values, a row's pairs by its four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t t;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
  return t;
}

template <int D, int NT>
struct Shared {                           // at a 1024-byte boundary: the tiles' swizzle pattern
  uint8_t tile[kWarpsOf<NT>][kTileSlots<D, NT>][kBlk * D];
  Entry ring[kWarpsOf<NT>][kRing];
  uint64_t full[kWarpsOf<NT>][kTileSlots<D, NT>];
  int64_t before[kWarpsOf<NT> * 32 + 1];  // visits before each thread's requests
  int64_t warp_sum[kWarpsOf<NT>];
};

template <int D, int NT>
constexpr int kSharedBytes = sizeof(Shared<D, NT>) + 1024;

// Whole warp: the phase of `bar` has completed, within the time limit.
__device__ __forceinline__ bool tile_ready(uint64_t* bar, uint32_t phase, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
  return mbar_wait_bounded_warp(bar, phase, kWaitNs, status);
}

}  // namespace

// One warp: thread (g, c) = (lane / 4, lane % 4).  K codes: thread c takes d in [32c,
// 32c + 32) (16c at d = 64) of keys 16i + g and 16i + g + 8, so the MMA's k indices
// stand for a permutation of d that q follows.  V codes: thread (g, c) takes d in
// [16g, 16g + 16) (8g) of keys 16i + {2c, 2c+1, 2c+8, 2c+9}; rows g and g + 8 of output
// tile t stand for d = 16g + 2t and + 1.  Both read patterns are free of bank conflicts
// in the swizzle of the tiles (two-way for V at d = 64).  The thread holds scores and
// outputs of rows 2c and 2c + 1 of each column block.
template <int D, bool kInt8, int NT>
__global__ void __launch_bounds__(kWarpsOf<NT> * 32, 1)
    q8_decode_kernel(const __grid_constant__ Q8Params p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, Q8Scratch scratch) {
  constexpr int kWarps = kWarpsOf<NT>, kRows = 8 * NT;
  constexpr int kSlots = kTileSlots<D, NT>;
  constexpr int kSteps = D / 16;          // k-steps of S
  constexpr int kOut = D / 16;            // output tiles
  constexpr int kPer = D / 4;             // q values of a thread and row
  constexpr int kCols = D / 8;            // output values of a thread and row
  extern __shared__ uint8_t raw[];
  Shared<D, NT>& sm = *reinterpret_cast<Shared<D, NT>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();

  if (tid < kWarps * kSlots) mbar_init1(&sm.full[tid / kSlots][tid % kSlots]);
  if (tid == 0) {
    prefetch_map(&k_map);
    prefetch_map(&v_map);
  }
  // Visits before each thread's share of the requests.
  const int share = (p.batch + kWarps * 32 - 1) / (kWarps * 32);
  int64_t mine = 0;
  for (int r = tid * share; r < min(p.batch, (tid + 1) * share); ++r) {
    mine += visits_of<NT>(p, r);
    if (blockIdx.x == 0) {
      bool bad;
      const Q8Request x = q8_request(p, r, &bad);
      if (bad) report_status(p.status, kStatusBadSchedule);
      if (x.n > 0 && (x.len + kBlk - 1) / kBlk > p.max_blocks) report_status(p.status, kStatusBadBlockTable);
    }
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  mbar_init_fence();
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  sm.before[tid] = base + incl - mine;
  if (tid == 0) sm.before[kWarps * 32] = total;
  __syncthreads();

  const int parts = gridDim.x * kWarps;
  const int part = warp * gridDim.x + blockIdx.x;   // neighbours in the list go to different SMs
  int64_t len = (total + parts - 1) / parts;
  if (len < kQ8MinVisits) len = kQ8MinVisits;
  const int64_t v0 = part * len, v1 = min(v0 + len, total);
  int* meta = scratch.meta + (size_t)part * 8;
  if (v0 >= v1) {
    if (lane == 0) meta[0] = 0;
    return;
  }
  Cursor<NT> cur;
  {
    int lo = 0, hi = kWarps * 32 - 1;               // the last share that starts at or before v0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sm.before[mid] <= v0) lo = mid;
      else hi = mid - 1;
    }
    cur.r = lo * share;
    cur.seek(p, v0 - sm.before[lo]);
  }
  const int visits = (int)(v1 - v0);
  Entry* ring = sm.ring[warp];
  uint64_t* full = sm.full[warp];
  const uint32_t tiles = smem_u32(&sm.tile[warp][0][0]);

  // The loading side runs ahead of the computing one by the ring's tiles.  It
  // reads the table and the scales of up to 32 visits of a request at a time.
  Cursor<NT> ahead = cur;
  int known = 0;                                    // visits whose entries are in the ring
  auto fill_ring = [&]() {
    const int64_t left = (int64_t)(ahead.units - ahead.unit) * ahead.count - ahead.blk;
    const int m = (int)min((int64_t)min(32, visits - known), left);
    if (lane < m) {
      const int at = ahead.blk + lane;
      const int unit = ahead.unit + at / ahead.count;
      const int blk = ahead.first + at % ahead.count;
      Entry e{-1, unit % p.h_kv, 0.f, 0.f};
      if (blk < p.max_blocks && blk * (int64_t)kBlk < ahead.x.len) {
        const int page = p.block_table[(int64_t)ahead.r * p.max_blocks + blk];
        if (page >= 0 && page < p.num_blocks) {
          e.block = page;
          e.k_scale = p.k_scale[page * p.k_scale_stride + e.head];
          e.v_scale = p.v_scale[page * p.v_scale_stride + e.head];
        } else {
          report_status(p.status, kStatusBadBlockTable);
        }
      }
      ring[(known + lane) % kRing] = e;
    }
    known += m;
    const int64_t at = ahead.blk + m;
    ahead.unit += (int)(at / ahead.count);
    ahead.blk = (int)(at % ahead.count);
    if (ahead.unit >= ahead.units && known < visits) ahead.next_request(p);
    __syncwarp();
  };
  auto issue = [&](int tile, int slot) {            // tile 2v: keys of visit v, 2v + 1: values
    const int v = tile >> 1;
    if (v >= visits) return;
    while (v >= known) fill_ring();
    if (lane == 0) {
      const Entry e = ring[v % kRing];
      if (e.block >= 0) {
        mbar_arrive_tx(&full[slot], kBlk * D);
        tma_tile(tiles + slot * (kBlk * D), (tile & 1) ? &v_map : &k_map, e.head, e.block, &full[slot]);
      } else {
        mbar_arrive1(&full[slot]);
      }
    }
  };
  for (int i = 0; i < kSlots; ++i) issue(i, i);

  uint32_t Q[NT][kSteps][2];
  float O[NT][kOut][4];
  // of rows 2c and 2c + 1 of each column block: power of two of q, softmax state, visibility
  float row_fac[NT][2], m[NT][2], l[NT][2], slope[NT][2], pos[NT][2];
  int lo[NT][2], hi[NT][2], all_lo = 0, all_hi = 0;
  float base_log2 = 0.f;
  bool opened = false;                              // base_log2 is set
  const float sl2 = p.scale * kLog2e;

  auto open_unit = [&]() {
    const int head = cur.unit % p.h_kv, rt = cur.unit / p.h_kv;
    opened = false;
    all_lo = 0;
    all_hi = 0x7FFFFFFF;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      {                                             // q of row 8 nt + g
        const int row = rt * kRows + 8 * nt + g, t = row / p.group, hq = head * p.group + row % p.group;
        uint4 w[kPer / 8];
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k) w[k] = make_uint4(0, 0, 0, 0);
        if (t < cur.x.n) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(cur.x.q0 + t) * p.q_token_stride +
                                                            (int64_t)hq * p.q_head_stride + kPer * c);
#pragma unroll
          for (int k = 0; k < kPer / 8; ++k) w[k] = __ldg(src + k);
        }
        auto lo_of = [](uint32_t v) { return __uint_as_float(v << 16); };
        auto hi_of = [](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); };
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k) {
          const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max3(top, fabsf(lo_of(u[j])), fabsf(hi_of(u[j])));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        row_pow2(top, up, down);
#pragma unroll
        for (int i = 0; i < 2; ++i) row_fac[nt][i] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + i));
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint4 a = w[s >> 1];
          const uint32_t x = s & 1 ? a.z : a.x, y = s & 1 ? a.w : a.y;
          Q[nt][s][0] = pack_f16(lo_of(x) * up, hi_of(x) * up);
          Q[nt][s][1] = pack_f16(lo_of(y) * up, hi_of(y) * up);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = rt * kRows + 8 * nt + 2 * c + i, t = row / p.group, hq = head * p.group + row % p.group;
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
        lo[nt][i] = 0;
        hi[nt][i] = 0x7FFFFFFF;
        slope[nt][i] = 0.f;
        pos[nt][i] = (float)(cur.x.len - cur.x.n + t);
        if (t < cur.x.n) {
          q8_visible(p, cur.x, t, lo[nt][i], hi[nt][i]);
          if (p.slopes) slope[nt][i] = p.slopes[hq] * kLog2e;
          all_lo = max(all_lo, lo[nt][i]);
          all_hi = min(all_hi, hi[nt][i]);
        }
      }
#pragma unroll
      for (int t = 0; t < kOut; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[nt][t][k] = 0.f;
    }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
  };

  // The unit's result, or this warp's piece of it.
  auto close_unit = [&](bool whole, bool begun_here) {
    const int head = cur.unit % p.h_kv, rt = cur.unit / p.h_kv;
    const float back = ex2(base_log2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s = l[nt][i];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const float inv = s == 0.f ? 0.f : back / s;
        const float lse2 = s == 0.f ? -INFINITY : m[nt][i] + log2f(s);
        const int in_tile = 8 * nt + 2 * c + i, row = rt * kRows + in_tile, t = row / p.group;
        const int hq = head * p.group + row % p.group;
        if (t >= cur.x.n) continue;
        // rows g and g + 8 of output tile k: d = kCols g + 2k and + 1
        if (whole) {
          const int64_t at = (int64_t)(cur.x.q0 + t) * p.h_q + hq;
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + kCols * g);
#pragma unroll
          for (int k = 0; k < kOut / 4; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              __nv_bfloat162 b = __floats2bfloat162_rn(O[nt][4 * k + j][i] * inv, O[nt][4 * k + j][2 + i] * inv);
              u[j] = *reinterpret_cast<uint32_t*>(&b);
            }
            dst[k] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (g == 0) p.lse[at] = lse2 * kLn2;
        } else {
          const int64_t slot = 2 * (int64_t)part + (begun_here ? 1 : 0);
          float4* dst = reinterpret_cast<float4*>(scratch.o + (slot * kPartRows + in_tile) * D + kCols * g);
#pragma unroll
          for (int k = 0; k < kOut / 2; ++k)
            dst[k] = make_float4(O[nt][2 * k][i] * inv, O[nt][2 * k][2 + i] * inv, O[nt][2 * k + 1][i] * inv,
                                 O[nt][2 * k + 1][2 + i] * inv);
          if (g == 0) scratch.lse[slot * kPartRows + in_tile] = lse2;
        }
      }
  };

  // Which parts share the unit this range begins inside, for the merge.
  if (lane == 0) {
    meta[0] = cur.blk > 0 ? 1 : 0;
    if (cur.blk > 0) {
      const int64_t u0 = v0 - cur.blk;
      meta[1] = (int)(u0 / len);
      meta[2] = (int)((u0 + cur.count - 1) / len);
      meta[3] = cur.x.q0;
      meta[4] = cur.x.n;
      meta[5] = cur.unit % p.h_kv;
      meta[6] = cur.unit / p.h_kv;
    }
  }

  int slot = 0;
  uint32_t phase = 0;
  bool begun_here = cur.blk == 0;
  open_unit();
  int v = 0;
  for (; v < visits; ++v) {
    const Entry e = ring[v % kRing];
    const int j0 = (cur.first + cur.blk) * kBlk;
    // ---- S^T = K Q^T
    if (!tile_ready(&full[slot], phase, p.status)) break;
    float S[NT][4][4];                              // [16 keys][key g: rows 2c, 2c + 1; key g + 8: the same]
    if (e.block >= 0) {
      const uint32_t kt = tiles + slot * (kBlk * D) + g * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[2][D / 16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t row = kt + (16 * i + 8 * h) * D;
          const uint4 a = lds128(row + (D == 128 ? ((2 * c) ^ g) << 4 : (c ^ ((g >> 1) & 3)) << 4));
          w[h][0] = a.x, w[h][1] = a.y, w[h][2] = a.z, w[h][3] = a.w;
          if constexpr (D == 128) {
            const uint4 b = lds128(row + (((2 * c + 1) ^ g) << 4));
            w[h][4] = b.x, w[h][5] = b.y, w[h][6] = b.z, w[h][7] = b.w;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt][i][0] = S[nt][i][1] = S[nt][i][2] = S[nt][i][3] = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t a0, a1, a2, a3;
          Q8Codes<kInt8>::to_f16(w[0][s], a0, a2);
          Q8Codes<kInt8>::to_f16(w[1][s], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(S[nt][i], a0, a1, a2, a3, Q[nt][s][0], Q[nt][s][1]);
        }
      }
    }
    __syncwarp();
    issue(2 * v + kSlots, slot);
    if (++slot == kSlots) slot = 0, phase ^= 1;
    // ---- softmax
    uint32_t P[NT][4][2];                           // [16 keys][keys 2c, 2c + 1 and + 8 of row g]
    if (e.block >= 0) {
      if (!opened) {
        base_log2 = e.v_scale > 0.f ? log2f(e.v_scale) : 0.f;
        opened = true;
      }
      const float rel = rel_log2(e.v_scale, base_log2), unrel = ex2(-rel);
      const bool edge = j0 < all_lo || j0 + kBlk > all_hi;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = row_fac[nt][i] * e.k_scale * sl2;
          if (p.cap > 0.f) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = S[nt][j >> 1][2 * (j & 1) + i];
            cap_scores<8>(x, f * p.inv_cap_log2, p.cap_log2);
#pragma unroll
            for (int j = 0; j < 8; ++j) S[nt][j >> 1][2 * (j & 1) + i] = x[j];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) S[nt][j >> 1][2 * (j & 1) + i] *= f;
          }
          if (p.slopes) {
            const float d0 = pos[nt][i] - (float)(j0 + g);
#pragma unroll
            for (int j = 0; j < 8; ++j) S[nt][j >> 1][2 * (j & 1) + i] -= slope[nt][i] * fabsf(d0 - (float)(8 * j));
          }
          if (edge) {
            const int a = lo[nt][i] - j0 - g, b = hi[nt][i] - j0 - g;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (8 * j < a || 8 * j >= b) S[nt][j >> 1][2 * (j & 1) + i] = -INFINITY;
          }
        }
      }
      float top[NT][2];
      bool grew = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a = fmaxf(S[nt][0][i], S[nt][0][2 + i]);
#pragma unroll
          for (int j = 1; j < 4; ++j) a = max3(a, S[nt][j][i], S[nt][j][2 + i]);
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
          top[nt][i] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16)) + rel;
          grew |= top[nt][i] > m[nt][i] + 8.f;
        }
      // P may grow to 2^8 before the accumulators are rescaled (f16 reaches 2^15)
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float now = fmaxf(m[nt][i], top[nt][i]);
            const float a = now == -INFINITY ? 1.f : ex2(m[nt][i] - now);
            m[nt][i] = now;
            l[nt][i] *= a;
#pragma unroll
            for (int t = 0; t < kOut; ++t) {
              O[nt][t][i] *= a;
              O[nt][t][2 + i] *= a;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float sub[2], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) sub[i] = m[nt][i] == -INFINITY ? 0.f : rel - m[nt][i];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = ex2(S[nt][j >> 1][2 * (j & 1)] + sub[0]), b = ex2(S[nt][j >> 1][2 * (j & 1) + 1] + sub[1]);
          sum[0] += a;
          sum[1] += b;
          P[nt][j >> 1][j & 1] = transpose8(pack_f16(a, b));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) l[nt][i] = fmaf(sum[i], unrel, l[nt][i]);
      }
    }
    // ---- O^T += V^T P^T
    if (!tile_ready(&full[slot], phase, p.status)) break;
    const uint32_t vt = tiles + slot * (kBlk * D);
    if (e.block >= 0) {
      const int tail = cur.x.len - j0;              // rows from here on are not the request's
      if (tail < kBlk) {                            // P is 0 there, and whatever they hold must not be a NaN
        for (int i = tail * (D / 16) + lane; i < kBlk * (D / 16); i += 32)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vt + 16 * i), "r"(0) : "memory");
        fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        uint32_t w[4][D / 32];                      // keys 16 kk + {2c, 2c+1, 2c+8, 2c+9}
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * kk + 2 * c + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 a = lds128(vt + row * D + ((g ^ (2 * c + (i & 1))) << 4));
            w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w;
          } else {
            const uint2 a = lds64(vt + row * D + (((g >> 1) ^ c) << 4) + ((g & 1) << 3));
            w[i][0] = a.x, w[i][1] = a.y;
          }
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q)            // output tiles 2q and 2q + 1
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            Q8Codes<kInt8>::to_f16(__byte_perm(w[0][q], w[1][q], h ? 0x7362 : 0x5140), a0, a1);
            Q8Codes<kInt8>::to_f16(__byte_perm(w[2][q], w[3][q], h ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(O[nt][2 * q + h], a0, a1, a2, a3, P[nt][kk][0], P[nt][kk][1]);
          }
      }
    }
    __syncwarp();
    issue(2 * v + 1 + kSlots, slot);
    if (++slot == kSlots) slot = 0, phase ^= 1;
    // ---- the end of a unit, or of the range
    const bool done = cur.blk + 1 == cur.count;
    if (done || v + 1 == visits) close_unit(done && begun_here, begun_here);
    if (v + 1 < visits) {
      cur.step(p);
      if (done) {
        begun_here = true;
        open_unit();
      }
    }
  }
  if (v < visits)                                   // a wait gave up: see the copies in flight out before leaving
    for (int i = 0; i < kSlots; ++i) {
      tile_ready(&full[slot], phase, p.status);
      if (++slot == kSlots) slot = 0, phase ^= 1;
    }
}

// Merges the pieces of a unit.  Part p whose range begins inside a unit that
// parts first .. last share merges the rows p - first - 1 + k (last - first).
template <int D, int NT>
__global__ void __launch_bounds__(128) q8_combine_kernel(const __grid_constant__ Q8Params p, Q8Scratch scratch) {
  __shared__ float acc[4][D];
  __shared__ float wsum[4];
  const int part = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait_primary();
  const int* meta = scratch.meta + (size_t)part * 8;
  if (meta[0] == 0) return;
  const int first = meta[1], last = meta[2], n = meta[4], rt = meta[6];
  constexpr int kRows = 8 * NT;
  const int rows = min(kRows, n * p.group - rt * kRows);
  constexpr int kV = D / 32;
  for (int row = part - first - 1; row < rows; row += last - first) {
    auto slot_of = [&](int q) { return (int64_t)2 * q + (q == first ? 1 : 0); };
    float top = -INFINITY;
    for (int q = first + lane; q <= last; q += 32) top = fmaxf(top, scratch.lse[slot_of(q) * kPartRows + row]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.f, o[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int q = first + warp; q <= last; q += 4) {
      const int64_t at = slot_of(q) * kPartRows + row;
      const float lse = scratch.lse[at];
      const float w = lse == -INFINITY ? 0.f : ex2(lse - top);
      const float* src = scratch.o + at * D + kV * lane;
      sum += w;
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] = fmaf(w, src[k], o[k]);
    }
    if (lane == 0) wsum[warp] = sum;
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[warp][kV * lane + k] = o[k];
    __syncthreads();
    const float all = wsum[0] + wsum[1] + wsum[2] + wsum[3];
    const int idx = rt * kRows + row, t = idx / p.group, hq = meta[5] * p.group + idx % p.group;
    const int64_t at = (int64_t)(meta[3] + t) * p.h_q + hq;
    const float inv = all == 0.f ? 0.f : 1.f / all;
    for (int i = threadIdx.x; i < D; i += 128)
      p.o[at * D + i] = __float2bfloat16((acc[0][i] + acc[1][i] + acc[2][i] + acc[3][i]) * inv);
    if (threadIdx.x == 0) p.lse[at] = (top == -INFINITY ? -INFINITY : top + log2f(all)) * kLn2;
    __syncthreads();
  }
}

namespace {

template <int D, bool kInt8, int NT>
cudaError_t launch(const Q8Params& p, const CUtensorMap& k_map, const CUtensorMap& v_map, const Q8Scratch& scratch,
                   int ctas, cudaStream_t stream) {
  constexpr int kWarps = kWarpsOf<NT>, kBytes = kSharedBytes<D, NT>;
  // per call: the attribute belongs to the current context and costs no launch
  if (const cudaError_t e = cudaFuncSetAttribute(q8_decode_kernel<D, kInt8, NT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
      e != cudaSuccess)
    return e;
  q8_decode_kernel<D, kInt8, NT><<<ctas, kWarps * 32, kBytes, stream>>>(p, k_map, v_map, scratch);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas * kWarps));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_combine_kernel<D, NT>, p, scratch);
}

template <int D, bool kInt8>
cudaError_t launch_rows(const Q8Params& p, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                        const Q8Scratch& scratch, int ctas, cudaStream_t stream) {
  return rows <= 8 ? launch<D, kInt8, 1>(p, k_map, v_map, scratch, ctas, stream)
                   : launch<D, kInt8, 2>(p, k_map, v_map, scratch, ctas, stream);
}

}  // namespace

cudaError_t launch_q8_decode(const Q8Params& p, bool int8, int rows, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, const Q8Scratch& scratch, int ctas, cudaStream_t stream) {
  if (p.d == 128)
    return int8 ? launch_rows<128, true>(p, rows, k_map, v_map, scratch, ctas, stream)
                : launch_rows<128, false>(p, rows, k_map, v_map, scratch, ctas, stream);
  return int8 ? launch_rows<64, true>(p, rows, k_map, v_map, scratch, ctas, stream)
              : launch_rows<64, false>(p, rows, k_map, v_map, scratch, ctas, stream);
}

}  // namespace smla
