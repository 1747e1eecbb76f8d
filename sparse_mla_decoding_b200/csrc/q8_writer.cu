// q8_writer.cu -- write new tokens into the block-scaled 8-bit cache.
//
// For each (block, head) that a call writes to, with `was` the block's scale if
// it holds older tokens of the request and 0 if it does not:
//   s    = the smallest power of two with max |x| / s <= 448 (e4m3) or 127 (int8)
//          over the new tokens' finite values; 0 if they are all zero
//   now  = max(s, was);  code = round-to-nearest-even(x / now), saturated
//   older codes become round(code * (was / now)) where now > was;
// for now = 0 all codes are 0 but those of NaN, which e4m3 keeps at any scale.
// Powers of two make x / s and the rescaling of e4m3 codes exact (up to the
// code's own rounding), and a block that fills token by token is rescaled only
// when its maximum crosses a power of two, not at every new maximum.  The price: a power
// of two lies up to 2x above the smallest scale that fits.  e4m3 has the exponent for it;
// of int8's codes up to half stay unused, so a value is off by up to twice the half step of
// the tightest scale, one bit of eight.
//
// One CTA per (block, head, keys or values): the block's new tokens stay in
// registers between the maximum and the codes, so everything is read and
// written once.  Bound by HBM for prompts (2 bytes read and 1 written a value),
// by latency for single tokens.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "q8_cache.h"
#include "q8_writer.h"
#include "sm100.cuh"

namespace smla {

namespace {

constexpr int kThreads = 128;

template <bool kInt8>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  if constexpr (kInt8) {
    // NaN becomes 0
    auto one = [](float x) { return (uint32_t)(__float2int_rn(fminf(fmaxf(x == x ? x : 0.f, -127.f), 127.f)) & 0xFF); };
    return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
}

template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
  if constexpr (kInt8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  } else {
    uint32_t lo, hi;
    Q8Codes<false>::to_f16(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  }
}

// The smallest power of two (at least 2^-126) at which amax fits the codes.
template <bool kInt8>
__device__ __forceinline__ float scale_for(float amax) {
  if (amax == 0.f) return 0.f;
  int e;
  const float m = frexpf(amax, &e);                          // m in [0.5, 1)
  const int k = kInt8 ? (m <= 127.f / 128.f ? e - 7 : e - 6)  // 127 = (127/128) 2^7
                      : (m <= 0.875f ? e - 9 : e - 8);        // 448 = 0.875 2^9
  return ldexpf(1.f, max(k, -126));
}

}  // namespace

// 64 registers, so that eight CTAs (128 KB of input) are under way on an SM.
template <int D, bool kInt8>
__global__ void __launch_bounds__(kThreads, 8) quantize_kv_blocks_kernel(const __grid_constant__ Q8WriteParams p) {
  constexpr int kLanes = D / 8;                  // threads of a row: 16 bytes of bf16 each
  constexpr int kAtOnce = kThreads / kLanes;     // rows in flight
  constexpr int kPasses = kBlk / kAtOnce;
  __shared__ float s_max[kThreads / 32];
  __shared__ int s_first, s_end, s_old, s_new;   // the request: its tokens, its lengths
  const int tid = threadIdx.x, x = blockIdx.x, head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  // Request r may touch the work items from cu[r] / 64 + 2r on: one more block than its
  // tokens fill at either end.  The owner is the last that starts at or before this
  // item; the thread that tests a request has its lengths ready for the others.
  int r = -1;
  for (int i0 = 0; i0 < p.batch; i0 += kThreads) {
    const int i = min(i0 + tid, p.batch - 1);
    const int a = p.cu[i], b = p.cu[i + 1], old = p.seqlens[i], now = p.new_seqlens[i];
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0 && (a < 0 || b < a || b > p.total || old < 0))
      report_status(p.status, kStatusBadSchedule);
    const bool before = i0 + tid < p.batch && (int64_t)(max(a, 0) / kBlk) + 2 * (int64_t)i <= x;
    const int c = __syncthreads_count(before);
    if (c > 0 && r == i0 - 1 && tid == c - 1) s_first = a, s_end = b, s_old = old, s_new = now;
    if (r == i0 - 1) r += c;
    if (c < kThreads && blockIdx.x + blockIdx.y + blockIdx.z > 0) break;   // the first CTA looks them all over
  }
  if (r < 0) return;
  __syncthreads();
  const int q0 = s_first, q1 = s_end, old = s_old;
  if (q0 < 0 || q1 < q0 || q1 > p.total || old < 0) return;
  const int n = q1 - q0;
  const int64_t item = x - (int64_t)(q0 / kBlk) - 2 * (int64_t)r;
  // a request that was not granted its blocks keeps its length: nothing to write
  if (n == 0 || item < 0 || (int64_t)s_new - old != n) return;
  const int64_t blk = old / kBlk + item;
  if (blk > ((int64_t)old + n - 1) / kBlk) return;
  const int row0 = (int)max((int64_t)old - blk * kBlk, (int64_t)0);            // first row written
  const int64_t t0 = blk * kBlk + row0 - old;                                 // its new token
  const int rows = (int)min((int64_t)kBlk - row0, n - t0);
  const int64_t stride = values ? p.v_token_stride : p.k_token_stride;
  const int sub = tid / kLanes, col = tid % kLanes;
  const __nv_bfloat16* src =
      (values ? p.v : p.k) + (q0 + t0 + sub) * stride + head * (values ? p.v_head_stride : p.k_head_stride) + 8 * col;
  uint4 w[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (sub + i * kAtOnce < rows) w[i] = __ldg(reinterpret_cast<const uint4*>(src + i * kAtOnce * stride));
  }
  // the tokens are on their way; where they go
  const int page = blk < p.max_blocks ? p.block_table[(int64_t)r * p.max_blocks + blk] : -1;
  if (page < 0 || page >= p.num_blocks) {
    if (tid == 0) report_status(p.status, kStatusBadBlockTable);
    return;
  }
  uint8_t* dst = (values ? p.v_cache + page * p.v_block_bytes : p.k_cache + page * p.k_block_bytes) +
                 (int64_t)head * kBlk * D;
  float* scale = (values ? p.v_scale + page * p.v_scale_stride : p.k_scale + page * p.k_scale_stride) + head;
  const float was = row0 > 0 ? *scale : 0.f;

  auto lo_of = [](uint32_t b) { return __uint_as_float(b << 16); };
  auto hi_of = [](uint32_t b) { return __uint_as_float(b & 0xFFFF0000u); };
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t b[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = fabsf(lo_of(b[j])), v = fabsf(hi_of(b[j]));
      if (u < INFINITY) amax = fmaxf(amax, u);
      if (v < INFINITY) amax = fmaxf(amax, v);
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float now = fmaxf(scale_for<kInt8>(amax), was);

  // older tokens of a block whose scale grew
  if (was < now) {
    const float ratio = was / now;
#pragma unroll 1
    for (int i = tid; i < row0 * (D / 4); i += kThreads) {
      float f[4];
      decode4<kInt8>(reinterpret_cast<uint32_t*>(dst)[i], f);
      reinterpret_cast<uint32_t*>(dst)[i] = code4<kInt8>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
    }
  }
  uint2* out = reinterpret_cast<uint2*>(dst + (row0 + sub) * D + 8 * col);
  if ((__float_as_uint(now) & 0x007FFFFFu) == 0u && now < 1.7e38f) {
    // a power of two (or 0) divides exactly by its inverse
    const float inv = now > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(now)) : 0.f;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      // all zeros, infinities beside zeros among them, for a zero scale
      const uint4 b = now > 0.f ? w[i] : make_uint4(0, 0, 0, 0);
      const uint2 c = make_uint2(code4<kInt8>(lo_of(b.x) * inv, hi_of(b.x) * inv, lo_of(b.y) * inv, hi_of(b.y) * inv),
                                 code4<kInt8>(lo_of(b.z) * inv, hi_of(b.z) * inv, lo_of(b.w) * inv, hi_of(b.w) * inv));
      if (sub + i * kAtOnce < rows) out[i * kAtOnce * (D / 8)] = c;
    }
  } else {
    // an older scale of some other kind: divide, reading the tokens again
#pragma unroll 1
    for (int i = sub; i < rows; i += kAtOnce)
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const float v = __fdiv_rn(__bfloat162float(src[(i - sub) * stride + j]), now);
        reinterpret_cast<uint8_t*>(out + (i - sub) * (D / 8))[j] = (uint8_t)code4<kInt8>(v, v, v, v);
      }
  }
  if (!kInt8 && now == 0.f) {
    // zeros and infinities, written above, and NaN (the tokens are read again: the registers
    // are the usual way's)
#pragma unroll 1
    for (int i = sub; i < rows; i += kAtOnce)
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const float x = __bfloat162float(src[(i - sub) * stride + j]);
        if (x != x) reinterpret_cast<uint8_t*>(out + (i - sub) * (D / 8))[j] = (uint8_t)code4<false>(x, x, x, x);
      }
  }
  if (tid == 0) *scale = now;
}

cudaError_t launch_q8_write(const Q8WriteParams& p, int d, bool int8, cudaStream_t stream) {
  const dim3 grid((unsigned)(p.total / kBlk + 2 * (int64_t)p.batch), (unsigned)p.h_kv, 2);
  if (d == 128) {
    if (int8) quantize_kv_blocks_kernel<128, true><<<grid, kThreads, 0, stream>>>(p);
    else quantize_kv_blocks_kernel<128, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (int8) quantize_kv_blocks_kernel<64, true><<<grid, kThreads, 0, stream>>>(p);
    else quantize_kv_blocks_kernel<64, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace smla
