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
// cut into equal ranges, one per CTA, and those into one per warp; a warp walks its
// range alone, with its own ring of TMA tiles, and no warp waits for another.  A
// range that holds a whole (request, tile, head) writes o itself; pieces of one are
// normalised partials in the workspace.  When its warps are done a CTA merges the
// pieces that it has of each unit (by their lse), so at most two partials a CTA are
// left for q8_combine_kernel.
//
// Products: S^T = K Q^T and O^T = V^T P^T on m16n8k16, so the cache's codes fill
// the 16-row side and a tile has 8 rows (one MMA column block) or 16 (two): a group
// of 8 heads wastes nothing, where rows on the 16-row side would double the
// products and the softmax.  The codes go to f16 in registers, once for all rows.
//
// Numbers: codes are exact in f16, and q is scaled by a power of two per row: its
// elements down to 2^-17 of the row's largest are exact too, smaller ones off by up to
// 2^-25 of it.  The scales multiply in fp32, exponentials are ex2.approx (2 units in
// the last place).  A value scale rides in the exponent,
//   p_j = 2^(x_j + log2 v_scale - m),
// so one accumulator holds blocks of different scales; the sum of the softmax
// takes the factor out again per block.  P is rounded to f16 once (2^-11), with m 7 to
// 15 below the row's largest exponent.
//
// Bound by HBM: d + 1/16 bytes a key, value and head; what has to keep up is the
// conversion, about 470 instructions a warp and block (16 KB at d = 128).  What costs
// beside it is code that runs once: a step of decoding reads more than L2 holds, so
// each launch fetches its instructions from memory again.  Every part is therefore
// kept to one copy (at 140 KB of code, merging a few rows took 11000 clocks).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "q8_attention.h"
#include "q8_cache.h"
#include "q8_tma.cuh"
#include "sm100.cuh"

namespace smla {

namespace {

constexpr int kPartRows = kQ8PartRows;    // rows of a partial slot
constexpr int kBatch = 16;                // visits whose table entries a warp reads at once
constexpr int kRing = 2 * kBatch;         // and keeps
constexpr uint64_t kWaitNs = 2000000000ull;

// Warps of a CTA (8 rows take 168 registers at d = 128 and 128 at d = 64, 16 rows up
// to 255) and tiles of a warp's ring.  About 100 KB of tiles are enough to cover
// memory's latency, and more in flight is slower: 64 x 8192 tokens at d = 128 took 172
// us with 12 warps of one tile, 180 with 14 of one, 185 with 12 of two; 37 ragged
// requests at d = 64 50 us with 16 warps of two tiles, 52 with three, 54 with 12 of four.
template <int D, int NT>
constexpr int kWarpsOf = NT == 2 ? 8 : D == 128 ? 12 : 16;
template <int D, int NT>
constexpr int kTileSlots = NT == 1 ? (D == 128 ? 1 : 2) : (D == 128 ? 2 : 3);

// One visit, as the loading side leaves it for the computing one.
struct Entry {
  int block, head;                        // cache block (-1: nothing to read) and KV head
  float k_scale, v_scale;
  int blk, rt;                            // block of the request, row tile
  int ends;                               // bits: first and last visit of its unit
  int request;                            // slot of its request's Work
};
constexpr int kRequests = 8;              // requests whose Work a warp keeps (a batch of entries has one)

// Blocks [first, first + count) that any row of the request sees; at least one,
// so that every request with new tokens gets its outputs written.
__device__ __forceinline__ void block_span(const Q8Params& p, const Q8Request& x, int& first, int& count) {
  int lo = 0, hi = x.len;
  if (p.docs && x.n <= kQ8SpanTokens) {
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

// A request's share of the list of visits: units (row tile, KV head) of `count` blocks.
struct Work {
  Q8Request x;
  int first, count, units;
};

template <int NT>
__device__ __forceinline__ Work work_of(const Q8Params& p, int r, bool* bad) {
  Work w;
  w.x = q8_request(p, r, bad);
  block_span(p, w.x, w.first, w.count);
  w.units = p.h_kv * row_tiles<NT>(p, w.x.n);
  return w;
}

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

// 4 bytes to shared memory, without waiting for them.
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// 8 x 8 f16 values, a row's pairs by its four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t t;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
  return t;
}

// What a warp holds of a unit that it does not hold whole: of the one that its range
// begins inside (head), and of the one that it begins and does not end (tail).
struct Piece {
  int there, ends;                        // it exists; the unit ends in it
  int q0, n, head, rt;
};

// Where a warp's loading side stands: its request, and the visit (unit, blk) of it that
// the next batch of entries starts with.  Kept in shared memory: it is used once in
// a batch, and the registers are the accumulators'.
struct Loader {
  Work work;
  int r, unit, blk, batches;
  uint32_t skip;                          // visits from the start of request r to the range's
};

template <int D, int NT>
struct Shared {                           // at a 1024-byte boundary: the tiles' swizzle pattern
  uint8_t tile[kWarpsOf<D, NT>][kTileSlots<D, NT>][kBlk * D];
  Entry ring[kWarpsOf<D, NT>][kRing];
  Work request[kWarpsOf<D, NT>][kRequests];
  uint64_t full[kWarpsOf<D, NT>][kTileSlots<D, NT>];
  uint32_t before[kWarpsOf<D, NT> * 32];     // visits before each thread's requests
  int64_t warp_sum[kWarpsOf<D, NT>];
  Piece head[kWarpsOf<D, NT>], tail[kWarpsOf<D, NT>];
  Loader loader[kWarpsOf<D, NT>];
  float2 bias[kWarpsOf<D, NT>][8 * NT];      // of a row: position, and slope in base 2
  int2 sees[kWarpsOf<D, NT>][8 * NT];        // positions that a row sees
};

template <int D, int NT>
constexpr int kSharedBytes = sizeof(Shared<D, NT>) + 1024;
static_assert(kSharedBytes<128, 1> <= 232448 && kSharedBytes<64, 1> <= 232448 && kSharedBytes<128, 2> <= 232448 &&
                  kSharedBytes<64, 2> <= 232448,
              "227 KB a CTA");

// Whole warp: the phase of `bar` has completed, within the time limit.
__device__ __forceinline__ bool tile_ready(uint64_t* bar, uint32_t phase, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase))) return true;
  return mbar_wait_bounded_warp(bar, phase, kWaitNs, status);
}

}  // namespace

// The merge of normalised pieces of a row by eight lanes, against a running maximum:
// a lane's values are d = 32 k + 4 (lane % 8) and the next three.  A piece is one trip
// to L2 (some thousand clocks while other CTAs still stream), so a warp takes four rows
// at once and has four pieces of each under way.
template <int D>
struct Merged {
  static constexpr int kV = D / 32, kAtOnce = 4;
  float top = -INFINITY, sum = 0.f;
  float4 o[kV];

  __device__ __forceinline__ Merged() {
#pragma unroll
    for (int k = 0; k < kV; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  static __device__ __forceinline__ void axpy(float4& y, float a, const float4& x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
  }

  // Pieces from, from + step, .. last; piece q is in slot 2q, the first of a unit that
  // begins in it in slot 2q + 1.
  __device__ __forceinline__ void add(const float* po, const float* plse, int from, int last, int step, int begins,
                                      int row, int lane8) {
#pragma unroll 1
    for (int p0 = from; p0 <= last; p0 += step * kAtOnce) {
      float lse[kAtOnce];
      float4 x[kAtOnce][kV];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int q = min(p0 + j * step, last);       // past the last: read it again, with no weight
        const int64_t at = ((int64_t)2 * q + (q == begins ? 1 : 0)) * kPartRows + row;
        lse[j] = plse[at];
#pragma unroll
        for (int k = 0; k < kV; ++k) x[j][k] = reinterpret_cast<const float4*>(po + at * D)[8 * k + lane8];
        if (p0 + j * step > last) lse[j] = -INFINITY;
      }
      float now = top;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) now = fmaxf(now, lse[j]);
      const float keep = now == -INFINITY ? 1.f : ex2(top - now);
      top = now;
      sum *= keep;
#pragma unroll
      for (int k = 0; k < kV; ++k) o[k] = make_float4(o[k].x * keep, o[k].y * keep, o[k].z * keep, o[k].w * keep);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (lse[j] == -INFINITY) continue;
        const float w = ex2(lse[j] - now);
        sum += w;
#pragma unroll
        for (int k = 0; k < kV; ++k) axpy(o[k], w, x[j][k]);
      }
    }
  }
  __device__ __forceinline__ float inverse() const { return sum == 0.f ? 0.f : 1.f / sum; }
  __device__ __forceinline__ float lse2() const { return sum == 0.f ? -INFINITY : top + log2f(sum); }

  // row `row` of the request's rows: o and lse
  __device__ __forceinline__ void store(const Q8Params& p, int q0, int head, int row, int lane8) const {
    const int t = row / p.group, hq = head * p.group + row - t * p.group;
    const int64_t at = (int64_t)(q0 + t) * p.h_q + hq;
    const float inv = inverse();
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      __nv_bfloat162 a = __floats2bfloat162_rn(o[k].x * inv, o[k].y * inv);
      __nv_bfloat162 b = __floats2bfloat162_rn(o[k].z * inv, o[k].w * inv);
      reinterpret_cast<uint2*>(p.o + at * D)[8 * k + lane8] =
          make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    }
    if (lane8 == 0) p.lse[at] = lse2() * kLn2;
  }
  // as a piece
  __device__ __forceinline__ void keep(float* po, float* plse, int64_t at, int lane8) const {
    const float inv = inverse();
#pragma unroll
    for (int k = 0; k < kV; ++k)
      reinterpret_cast<float4*>(po + at * D)[8 * k + lane8] =
          make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv);
    if (lane8 == 0) plse[at] = lse2();
  }
};

// One warp: thread (g, c) = (lane / 4, lane % 4).  K codes: thread c takes d in [32c,
// 32c + 32) (16c at d = 64) of keys 16i + g and 16i + g + 8, so the MMA's k indices
// stand for a permutation of d that q follows.  V codes: thread (g, c) takes d in
// [16g, 16g + 16) (8g) of keys 16i + {2c, 2c+1, 2c+8, 2c+9}; rows g and g + 8 of output
// tile t stand for d = 16g + 2t and + 1.  Both read patterns are free of bank conflicts
// in the swizzle of the tiles (two-way for V at d = 64).  The thread holds scores and
// outputs of rows 2c and 2c + 1 of each column block.
template <int D, bool kInt8, int NT>
__global__ void __launch_bounds__(kWarpsOf<D, NT> * 32, 1)
    q8_decode_kernel(const __grid_constant__ Q8Params p, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, Q8Scratch scratch) {
  constexpr int kWarps = kWarpsOf<D, NT>, kRows = 8 * NT;
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
#pragma unroll 1
  for (int r = tid * share; r < min(p.batch, (tid + 1) * share); ++r) {
    bool bad;
    const Work w = work_of<NT>(p, r, &bad);
    mine += (int64_t)w.units * w.count;
    if (blockIdx.x == 0) {
      if (bad) report_status(p.status, kStatusBadSchedule);
      if (w.x.n > 0 && (w.x.len + kBlk - 1) / kBlk > p.max_blocks) report_status(p.status, kStatusBadBlockTable);
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
  int64_t base = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += sm.warp_sum[w];
    all += sm.warp_sum[w];
  }
  sm.before[tid] = (uint32_t)(base + incl - mine);
  __syncthreads();
  // 2^31 blocks are tens of TB to read: lengths that ask for more are not meant
  const uint32_t total = all < 0x7FFFFFFF ? (uint32_t)all : 0u;
  if (all >= 0x7FFFFFFF && blockIdx.x == 0 && tid == 0) report_status(p.status, kStatusBadSchedule);

  // The CTA's range of visits, and the warp's of it.
  const uint32_t cta_len = max((total + gridDim.x - 1) / gridDim.x, (uint32_t)kQ8MinVisits);
  const uint32_t len = (cta_len + kWarps - 1) / kWarps;
  const uint32_t c0 = min(blockIdx.x * cta_len, total), c1 = min(c0 + cta_len, total);
  const uint32_t v0 = min(c0 + warp * len, c1), v1 = min(v0 + len, c1);
  const int part = blockIdx.x * kWarps + warp, visits = (int)(v1 - v0);
  if (lane == 0) sm.head[warp].there = sm.tail[warp].there = 0;
  if (tid == 0) scratch.meta[(size_t)blockIdx.x * 8] = 0;
  Entry* ring = sm.ring[warp];
  uint64_t* full = sm.full[warp];
  const uint32_t tiles = smem_u32(&sm.tile[warp][0][0]);

  int known = 0;                                    // visits that have entries
  if (visits > 0) {
    int n = 0;                                      // shares that start at or before v0
#pragma unroll 1
    for (int i = 0; i < kWarps; ++i) n += sm.before[32 * i + lane] <= v0 ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n) - 1;      // the last of them (empty ones before it start there too)
    if (lane == 0) {
      Loader& at = sm.loader[warp];
      at.work.units = at.unit = at.blk = at.batches = 0;
      at.r = n * share - 1;
      at.skip = v0 - sm.before[n];
    }
    __syncwarp();
  }
  // A batch of entries: visits of one request.
  auto fill_ring = [&]() {
    Loader& state = sm.loader[warp];
    Work ahead = state.work;
    int r = state.r, unit = state.unit, blk = state.blk;
    const int batches = state.batches;
    uint32_t skip = state.skip;
    while (unit >= ahead.units) {                   // the next request that has visits
      ++r;
      bool bad;
      ahead = work_of<NT>(p, r, &bad);
      const uint32_t have = (uint32_t)ahead.units * (uint32_t)ahead.count, jump = min(skip, have);
      skip -= jump;
      unit = (int)(jump / (uint32_t)ahead.count);
      blk = (int)(jump - (uint32_t)unit * (uint32_t)ahead.count);
    }
    const uint32_t left = (uint32_t)(ahead.units - unit) * (uint32_t)ahead.count - (uint32_t)blk;
    const int m = (int)min((uint32_t)min(kBatch, visits - known), left);
    if (lane == 0) sm.request[warp][batches % kRequests] = ahead;
    const uint32_t at = (uint32_t)(blk + lane), up = at / (uint32_t)ahead.count, in_unit = at - up * ahead.count;
    if (lane < m) {
      const int u = unit + (int)up, rt = u / p.h_kv, head = u - rt * p.h_kv, b = ahead.first + (int)in_unit;
      Entry& e = ring[(known + lane) % kRing];
      int page = -1;
      if (b < p.max_blocks && b * (int64_t)kBlk < ahead.x.len) {
        page = p.block_table[(int64_t)r * p.max_blocks + b];
        if (page < 0 || page >= p.num_blocks) {
          report_status(p.status, kStatusBadBlockTable);
          page = -1;
        }
      }
      e.block = page;
      e.head = head;
      e.blk = b;
      e.rt = rt;
      e.ends = (in_unit == 0 ? 1 : 0) | ((int)in_unit + 1 == ahead.count ? 2 : 0);
      e.request = batches % kRequests;
      if (page >= 0) {                              // the copies of the tiles need not wait for these
        copy4(&e.k_scale, p.k_scale + page * p.k_scale_stride + head);
        copy4(&e.v_scale, p.v_scale + page * p.v_scale_stride + head);
      }
    }
    // For the combine kernel: which CTAs share the unit that this CTA's range begins inside.
    if (known == 0 && warp == 0 && lane == 0 && blk > 0) {
      int* meta = scratch.meta + (size_t)blockIdx.x * 8;
      const uint32_t u0 = v0 - (uint32_t)blk;
      meta[0] = 1;
      meta[1] = (int)(u0 / cta_len);
      meta[2] = (int)((u0 + (uint32_t)ahead.count - 1) / cta_len);
      meta[3] = ahead.x.q0;
      meta[4] = ahead.x.n;
      meta[5] = unit % p.h_kv;
      meta[6] = unit / p.h_kv;
    }
    known += m;
    __syncwarp();
    if (lane == 0) {
      const uint32_t next = (uint32_t)(blk + m), over = next / (uint32_t)ahead.count;
      state = {ahead, r, unit + (int)over, (int)(next - over * (uint32_t)ahead.count), batches + 1, skip};
    }
    __syncwarp();
  };
  // tile 2v: keys of visit v, 2v + 1: values
  auto issue = [&](int tile, int slot) {
    const int v = tile >> 1;
    if (v < visits && lane == 0) {
      const int block = ring[v % kRing].block, head = ring[v % kRing].head;
      if (block >= 0) {
        mbar_arrive_tx(&full[slot], kBlk * D);
        tma_tile(tiles + slot * (kBlk * D), (tile & 1) ? &v_map : &k_map, head, block, &full[slot]);
      } else {
        mbar_arrive1(&full[slot]);
      }
    }
  };

  uint32_t Q[NT][kSteps][2];
  float O[NT][kOut][4];
  // of rows 2c and 2c + 1 of each column block: power of two of q, softmax state
  float row_fac[NT][2], m[NT][2], l[NT][2];
  int all_lo = 0, all_hi = 0;                       // what every row of the tile sees
  float base_log2 = -INFINITY;                      // log2 of the unit's first value scale above 0
  const float sl2 = p.scale * kLog2e;
  // Token of row j of row tile rt, and its head in the group.  The division by the
  // group is by its inverse: exact below 2^20.
  auto token_of = [&](int rt, int j, int& in_group) {
    const int t0 = rt * kRows / p.group, h = rt * kRows - t0 * p.group + j;
    const int up = __float2int_rz(((float)h + 0.5f) * p.inv_group);
    in_group = h - up * p.group;
    return t0 + up;
  };

  // The unit's result, or this warp's piece of it.
  auto close_unit = [&](const Entry& e, const Q8Request& x, bool whole, bool begun_here) {
    const float back = exp2f(base_log2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s = l[nt][i];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        // the scale apart from 1 / s: for values of 2^-100 their product would lose bits
        const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
        for (int k = 0; k < kOut; ++k) O[nt][k][i] *= inv, O[nt][k][2 + i] *= inv;
        const float lse2 = s == 0.f ? -INFINITY : lse_log2(m[nt][i], s);
        const int in_tile = 8 * nt + 2 * c + i;
        int hh;
        const int t = token_of(e.rt, in_tile, hh), hq = e.head * p.group + hh;
        if (t >= x.n) continue;
        // rows g and g + 8 of output tile k: d = kCols g + 2k and + 1
        if (whole) {                                  // no visible key: 0, though a NaN value may be in O
          const int64_t at = (int64_t)(x.q0 + t) * p.h_q + hq;
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + kCols * g);
#pragma unroll
          for (int k = 0; k < kOut / 4; ++k) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              __nv_bfloat162 b = __floats2bfloat162_rn(O[nt][4 * k + j][i] * back, O[nt][4 * k + j][2 + i] * back);
              u[j] = s == 0.f ? 0u : *reinterpret_cast<uint32_t*>(&b);
            }
            dst[k] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (g == 0) p.lse[at] = lse2 * kLn2;
        } else {
          const int64_t slot = 2 * (int64_t)part + (begun_here ? 1 : 0);
          float4* dst = reinterpret_cast<float4*>(scratch.o + (slot * kPartRows + in_tile) * D + kCols * g);
#pragma unroll
          for (int k = 0; k < kOut / 2; ++k)
            dst[k] = make_float4(O[nt][2 * k][i] * back, O[nt][2 * k][2 + i] * back, O[nt][2 * k + 1][i] * back,
                                 O[nt][2 * k + 1][2 + i] * back);
          if (g == 0) scratch.lse[slot * kPartRows + in_tile] = lse2;
        }
      }
  };

  constexpr int kLead = (kSlots + 1) / 2;           // visits that the ring of tiles runs ahead
  int slot = 0, v = 0;
  uint32_t phase = 0;
  bool begun_here = false;
  for (; v < visits; ++v) {
    while (known < min(visits, v + 1 + kLead)) fill_ring();
    if (v == 0) {
#pragma unroll 1
      for (int i = 0; i < kSlots; ++i) issue(i, i);
    }
    const int ends = ring[v % kRing].ends;
    if (v == 0 || (ends & 1)) {                     // open a unit
      const int head = ring[v % kRing].head, rt = ring[v % kRing].rt;
      const Q8Request x = sm.request[warp][ring[v % kRing].request].x;
      begun_here = ends & 1;
      base_log2 = -INFINITY;
      all_lo = 0;
      all_hi = 0x7FFFFFFF;
      uint4 raw_q[NT][kPer / 8];                    // q of row 8 nt + g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        int hh;
        const int t = token_of(rt, 8 * nt + g, hh);
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k) raw_q[nt][k] = make_uint4(0, 0, 0, 0);
        if (t < x.n) {
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (int64_t)(x.q0 + t) * p.q_token_stride + (int64_t)(head * p.group + hh) * p.q_head_stride +
              kPer * c);
#pragma unroll
          for (int k = 0; k < kPer / 8; ++k) raw_q[nt][k] = __ldg(src + k);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          int hh;
          const int t = token_of(rt, 8 * nt + 2 * c + i, hh);
          m[nt][i] = -INFINITY;
          l[nt][i] = 0.f;
          int lo = 0, hi = 0x7FFFFFFF;
          float2 bias = make_float2(0.f, 0.f);      // an absent row's scores are 0, and its vote always the same
          if (t < x.n) {
            q8_visible(p, x, t, lo, hi);
            if (p.slopes) bias = make_float2((float)(x.len - x.n + t), p.slopes[head * p.group + hh] * kLog2e);
            all_lo = max(all_lo, lo);
            all_hi = min(all_hi, hi);
          }
          if (g == 0) {
            sm.sees[warp][8 * nt + 2 * c + i] = make_int2(lo, hi);
            sm.bias[warp][8 * nt + 2 * c + i] = bias;
          }
        }
#pragma unroll
        for (int t = 0; t < kOut; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) O[nt][t][k] = 0.f;
      }
      all_lo = __reduce_max_sync(0xffffffffu, all_lo);
      all_hi = __reduce_min_sync(0xffffffffu, all_hi);
      auto lo_of = [](uint32_t b) { return __uint_as_float(b << 16); };
      auto hi_of = [](uint32_t b) { return __uint_as_float(b & 0xFFFF0000u); };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kPer / 8; ++k) {
          const uint32_t b[4] = {raw_q[nt][k].x, raw_q[nt][k].y, raw_q[nt][k].z, raw_q[nt][k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max3(top, fabsf(lo_of(b[j])), fabsf(hi_of(b[j])));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float up, down;
        row_pow2(top, up, down);
#pragma unroll
        for (int i = 0; i < 2; ++i) row_fac[nt][i] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + i));
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const uint4 a = raw_q[nt][s >> 1];
          const uint32_t b0 = s & 1 ? a.z : a.x, b1 = s & 1 ? a.w : a.y;
          Q[nt][s][0] = pack_f16(lo_of(b0) * up, hi_of(b0) * up);
          Q[nt][s][1] = pack_f16(lo_of(b1) * up, hi_of(b1) * up);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // the scales of the entries
    __syncwarp();
    // at d = 128 read where used: the registers are the accumulators'
    const std::conditional_t<D == 64, Entry, Entry&> e = ring[v % kRing];
    const int j0 = e.blk * kBlk;
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
      if (base_log2 == -INFINITY) base_log2 = log2f(e.v_scale);
      const float rel = rel_log2(e.v_scale, base_log2), unrel = ex2(-rel);
      const bool edge = j0 < all_lo || j0 + kBlk > all_hi;
      if (p.cap > 0.f && sm.request[warp][e.request].x.len - j0 < kBlk) {
        // what stands behind the length has no vote on the cap's form
        const int tail = sm.request[warp][e.request].x.len - j0 - g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (8 * j >= tail) S[nt][j >> 1][2 * (j & 1)] = S[nt][j >> 1][2 * (j & 1) + 1] = 0.f;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = fminf(row_fac[nt][i] * e.k_scale * sl2, kMostFactor);
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
            const float2 b = sm.bias[warp][8 * nt + 2 * c + i];
            const float d0 = b.x - (float)(j0 + g);
#pragma unroll
            for (int j = 0; j < 8; ++j) S[nt][j >> 1][2 * (j & 1) + i] -= b.y * fabsf(d0 - (float)(8 * j));
          }
          if (edge) {
            const int2 see = sm.sees[warp][8 * nt + 2 * c + i];
            const int a = see.x - j0 - g, b = see.y - j0 - g;
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
          grew |= top[nt][i] > m[nt][i] + (kHead + kLag);
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float now = fmaxf(m[nt][i], top[nt][i] - kHead);
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
      const int tail = sm.request[warp][e.request].x.len - j0;              // rows from here on are not the request's
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
    const bool done = e.ends & 2;
    if (done || v + 1 == visits) {
      const Q8Request x = sm.request[warp][e.request].x;
      close_unit(e, x, done && begun_here, begun_here);
      if (lane == 0 && !(done && begun_here))
        (begun_here ? sm.tail : sm.head)[warp] = {1, done ? 1 : 0, x.q0, x.n, e.head, e.rt};
    }
  }
  if (v < visits)                                   // a wait gave up: see the copies in flight out before leaving
    for (int i = 0; i < kSlots; ++i) {
      tile_ready(&full[slot], phase, p.status);
      if (++slot == kSlots) slot = 0, phase ^= 1;
    }

  // ---- merge what the CTA has of each unit, the rows of all units over the warps.  A
  // chain of pieces starts at a tail, or at the head of warp 0.
  __syncthreads();
  int turn = 0;
#pragma unroll 1
  for (int s = -1; s < kWarps; ++s) {
    const bool begun = s >= 0;
    const Piece& start = begun ? sm.tail[s] : sm.head[0];
    if (!start.there) continue;
    const int first = begun ? s : 0;
    int last = first;
    while (last + 1 < kWarps && ((begun && last == first) || !sm.head[last].ends) && sm.head[last + 1].there) ++last;
    const bool ended = begun && last == first ? false : sm.head[last].ends != 0;
    const int rows = min(kRows, start.n * p.group - start.rt * kRows);
    const int p0 = blockIdx.x * kWarps + first, p1 = blockIdx.x * kWarps + last;
#pragma unroll 1
    for (int row0 = 0; row0 < rows; row0 += 4) {
      const int row = row0 + (lane >> 3);
      if (turn++ % kWarps != warp || row >= rows) continue;
      Merged<D> got;
      got.add(scratch.o, scratch.lse, p0, p1, 1, begun ? p0 : -1, row, lane & 7);
      if (begun && ended)
        got.store(p, start.q0, start.head, start.rt * kRows + row, lane & 7);
      else
        got.keep(scratch.cta_o, scratch.cta_lse, (2 * (int64_t)blockIdx.x + (begun ? 1 : 0)) * kPartRows + row,
                 lane & 7);
    }
  }
}

// Merges what the CTAs have of a unit.  CTA c of the decode whose range begins inside
// a unit that CTAs first .. last share merges the rows c - first - 1 + k (last -
// first), so a long request's pieces are merged by as many CTAs as it has rows: eight
// lanes a row, or with a single row its pieces over all lanes.
constexpr int kCombineWarps = 4;

template <int D, int NT>
__global__ void __launch_bounds__(32 * kCombineWarps) q8_combine_kernel(const __grid_constant__ Q8Params p,
                                                                        Q8Scratch scratch) {
  constexpr int kRows = 8 * NT, kV = D / 32, kTeams = 4 * kCombineWarps;   // teams of eight lanes
  __shared__ float4 s_o[kTeams][D / 4];
  __shared__ float s_lse[kTeams];
  const int lane8 = threadIdx.x & 7, team = threadIdx.x >> 3;
  pdl_wait_primary();
  const int4* meta = reinterpret_cast<const int4*>(scratch.meta + (size_t)blockIdx.x * 8);
  const int4 ma = meta[0], mb = meta[1];
  if (ma.x == 0) return;
  const int first = ma.y, last = ma.z, q0 = ma.w, head = mb.y, rt = mb.z;
  const int rows = min(kRows, mb.x * p.group - rt * kRows);
  const int ctas = last - first, idx0 = blockIdx.x - first - 1;
  if (idx0 >= rows) return;
  const bool several = idx0 + ctas < rows;            // rows (at most 16: a team each)
  const int row = several ? idx0 + team * ctas : idx0;
  Merged<D> got;
  if (row < rows)
    got.add(scratch.cta_o, scratch.cta_lse, several ? first : first + team, last, several ? 1 : kTeams, first, row,
            lane8);
  if (several) {
    if (row < rows) got.store(p, q0, head, rt * kRows + row, lane8);
    return;
  }
  const float inv = got.inverse();
#pragma unroll
  for (int k = 0; k < kV; ++k)
    s_o[team][8 * k + lane8] = make_float4(got.o[k].x * inv, got.o[k].y * inv, got.o[k].z * inv, got.o[k].w * inv);
  if (lane8 == 0) s_lse[team] = got.lse2();
  __syncthreads();
  if (team == 0) {
    Merged<D> all;
    for (int w = 0; w < kTeams; ++w) all.top = fmaxf(all.top, s_lse[w]);
    for (int w = 0; w < kTeams; ++w) {
      if (s_lse[w] == -INFINITY) continue;
      const float f = ex2(s_lse[w] - all.top);
      all.sum += f;
#pragma unroll
      for (int k = 0; k < kV; ++k) Merged<D>::axpy(all.o[k], f, s_o[w][8 * k + lane8]);
    }
    all.store(p, q0, head, rt * kRows + row, lane8);
  }
}

namespace {

template <int D, bool kInt8, int NT>
cudaError_t launch(const Q8Params& p, const CUtensorMap& k_map, const CUtensorMap& v_map, const Q8Scratch& scratch,
                   int ctas, cudaStream_t stream) {
  constexpr int kWarps = kWarpsOf<D, NT>, kBytes = kSharedBytes<D, NT>;
  static SharedLimit limit;
  if (const cudaError_t e = raise_shared_limit(limit, (const void*)q8_decode_kernel<D, kInt8, NT>, kBytes);
      e != cudaSuccess)
    return e;
  q8_decode_kernel<D, kInt8, NT><<<ctas, kWarps * 32, kBytes, stream>>>(p, k_map, v_map, scratch);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q8_combine_kernel<D, NT>, p, scratch);
}

template <int D, bool kInt8>
cudaError_t launch_rows(const Q8Params& p, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                        const Q8Scratch& scratch, int ctas, cudaStream_t stream) {
  // 32 requests of 4096 tokens, 8 heads, with tiles of 8 and of 16 rows: at 8 rows 56 and 58
  // us (d = 64: 37 and 45), at 16 rows 84 and 61 (47 and 46), at 32 158 and 101 (79 and 76)
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
