// q8_cache.h -- what the kernels over the block-scaled 8-bit cache share: the
// launch parameters, the codes and their conversions, and the visibility rule.
//
// The cache holds keys and values in blocks of 64 tokens: codes
// [num_blocks][h_kv][64][d] in e4m3 or int8 and one float32 scale for each
// (block, head); a key is code * scale.  Row r of a request's n new tokens
// stands at position len - n + t of the request.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace smla {

constexpr int kBlk = 64;          // tokens per cache block
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMostFactor = 3e38f;   // of a score: finite, so that a product of 0 stays 0

// Everything an attention call over the cache needs; offsets and strides in
// elements unless they say bytes.
struct Q8Params {
  const __nv_bfloat16* q;         // [total_q][h_q][d]
  int64_t q_token_stride, q_head_stride;
  const float *k_scale, *v_scale; // [num_blocks][h_kv]
  int64_t k_scale_stride, v_scale_stride;
  const uint8_t *k_cache, *v_cache;
  int64_t k_block_bytes, v_block_bytes;
  int64_t num_blocks;
  const int32_t* block_table;     // [batch][max_blocks]
  const int32_t* seqlens;         // [batch], with the new tokens
  const int32_t* cu_q;            // [batch + 1], or NULL: s_q tokens each
  const float* slopes;            // [h_q] or NULL
  const int32_t* prefix;          // [batch] or NULL
  const int32_t* docs;            // [total_q][2] or NULL
  int max_blocks, batch, s_q, total_q, h_q, h_kv, group, d;
  int causal;
  float inv_group;                // 1 / group
  float scale;                    // softmax scale
  float cap;                      // 0: none
  float cap_log2, inv_cap_log2;   // cap log2(e) and its inverse
  __nv_bfloat16* o;               // [total_q][h_q][d]
  float* lse;                     // [total_q][h_q]
  uint32_t* status;               // may be NULL
};

// A request as the kernels see it.  n is 0 where the offsets are not usable.
struct Q8Request {
  int q0, n, len;                 // first row in q, new tokens, cache length
  int prefix;
};

__device__ __forceinline__ Q8Request q8_request(const Q8Params& p, int r, bool* bad) {
  Q8Request x;
  if (p.cu_q) {
    const int a = p.cu_q[r], b = p.cu_q[r + 1];
    const bool ok = a >= 0 && b >= a && b <= p.total_q;
    *bad = !ok;
    x.q0 = ok ? a : 0;
    x.n = ok ? b - a : 0;
  } else {
    *bad = false;
    x.q0 = r * p.s_q;
    x.n = p.s_q;
  }
  x.len = min(max(p.seqlens[r], 0), 0x7FFFFFFF - 256);   // the kernels round lengths up to blocks
  x.prefix = p.prefix ? p.prefix[r] : 0;
  return x;
}

// The cache positions [lo, hi) that new token t of a request sees, both >= 0: the kernels
// take positions off them.
__device__ __forceinline__ void q8_visible(const Q8Params& p, const Q8Request& x, int t, int& lo, int& hi) {
  lo = 0;
  hi = x.len;
  if (p.causal) hi = min(hi, max(x.len - x.n + t + 1, x.prefix));
  if (p.docs) {
    const int2 d = reinterpret_cast<const int2*>(p.docs)[x.q0 + t];
    lo = max(d.x, 0);
    hi = min(hi, d.y);
  }
  hi = max(hi, 0);
}

// ---------------------------------------------------------------------------
// codes -> f16: every e4m3 and int8 code is exact in f16 (4 and 8 significant
// bits; e4m3's range 2^-9 .. 448 lies inside f16's), so the matrix products see
// the cache's codes unrounded and the scales are applied in fp32.
// ---------------------------------------------------------------------------
template <bool kInt8>
struct Q8Codes;

template <>
struct Q8Codes<false> {
  // four codes of one word as two f16 pairs
  static __device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
};

template <>
struct Q8Codes<true> {
  // int8 + 128 as the low byte of 1024.0 (0x6400), then minus 1152: exact (a known way from
  // integers to floats; for 8-bit weights in f16 published by Kim et al., "Who says elephants
  // can't run", 2022).
  static __device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    lo = __byte_perm(w, 0x64646464u, 0x4140);
    hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), off);
    __half2 b = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
    lo = *reinterpret_cast<uint32_t*>(&a);
    hi = *reinterpret_cast<uint32_t*>(&b);
  }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 2^x, subnormal results flushed (a probability below 2^-126 of its row's
// largest): without the flush the compiler scales around every one of them.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The power of two that brings a row maximum `amax` into [1, 2) (as far as
// fp32's exponents reach), and its inverse.
__device__ __forceinline__ void row_pow2(float amax, float& up, float& down) {
  const int e = (int)(__float_as_uint(amax) >> 23) & 0xFF;
  const int k = min(max(e, 1), 253);
  up = __uint_as_float((uint32_t)(254 - k) << 23);
  down = __uint_as_float((uint32_t)k << 23);
}

// m + log2(s) of a softmax sum s > 0 to the reference m, which may both be far from 0 where
// value scales are (2^60, and zeros count as 2^-60): s's exponent joins m first, so that
// nothing is rounded at that size.
__device__ __forceinline__ float lse_log2(float m, float s) {
  float up, down;
  row_pow2(s, up, down);
  return m + (float)((int)(__float_as_uint(down) >> 23) - 127) + log2f(s * up);
}

// Two fp32 operations in one instruction; each is rounded as the scalar one.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The same, NaN where one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// x_j = cap tanh(x_j fc) of N scores; a vote of the warp over the N picks the way.
// All |y| = |x fc| <= 0.35: y P(y^2), P a degree-3 fit to tanh(y)/y in relative error
// (reweighted least squares on Chebyshev nodes; 1.5e-7 in fp32), so small scores keep
// their relative precision and no special function is used; fc and cap go into the
// coefficients, so a score costs 2.5 packed instructions.  Else 1 - 2 / (1 + exp(2
// |y|)) with the sign of x, off by some 1e-7 of the cap.  (x is a product of f16
// values, below 2^18, so x^2 stays in range; fc <= 2^9 keeps fc^7 cap, with caps up
// to 2^60, inside fp32, and a finite factor keeps 0 at 0.)
template <int N>
__device__ __forceinline__ void cap_scores(float* x, float fc, float cap) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < N; j += 2) top = max3(top, fabsf(x[j]), fabsf(x[j + 1]));
  if (__any_sync(0xffffffffu, !(top * fc <= 0.35f && fc <= 512.f))) {
    const float fe = fminf(fc * (2.f * kLog2e), kMostFactor);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(fabsf(x[j]) * fe)));
      x[j] = copysignf(fmaf(-2.f * cap, r, cap), x[j]);
    }
  } else {
    const float s = fc * fc, c0 = fc * cap, c1 = c0 * s, c2 = c1 * s;
    const float2 k0 = both(c0 * 0.9999999403953552f), k1 = both(c1 * -0.33332422375679016f),
                 k2 = both(c2 * 0.13295817375183105f), k3 = both(c2 * s * -0.04895907640457153f);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float2 v = make_float2(x[j], x[j + 1]), z = mul2(v, v);
      const float2 r = mul2(fma2(fma2(fma2(k3, z, k2), z, k1), z, k0), v);
      x[j] = r.x;
      x[j + 1] = r.y;
    }
  }
}

// The softmax reference m of a row lies kHead below its running maximum, so P = 2^(x - m)
// is 2^kHead there and, as m is raised only once the maximum is kHead + kLag above it, at
// most 2^15, inside f16.  f16 drops what is below 2^-25: keys of 2^-32 of the largest
// probability, of which a million weigh 2^-12, less than o's own rounding.
constexpr float kHead = 7.f, kLag = 8.f;

// log2 of a value scale relative to `base`, kept within 2^+-60 (a zero scale
// has only zero codes behind it, so any value does, and none is a base; the
// clamp keeps the softmax denominator inside fp32).
__device__ __forceinline__ float rel_log2(float scale, float base_log2) {
  return fminf(fmaxf(log2f(scale) - base_log2, -60.f), 60.f);
}

}  // namespace smla
