// q8_api.cu -- the C entries over the block-scaled 8-bit cache (declared in
// include/smla.h): argument checks, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/smla.h"
#include "q8_attention.h"
#include "q8_writer.h"
#include "splitkv_mla.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The largest |stride| or block count that keeps every product inside int64.
constexpr int64_t kMost = (int64_t)1 << 48;

int check_cache(const smla_q8_cache* c) {
  if (!c) return SMLA_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128) return SMLA_ERR_UNSUPPORTED;
  if (c->format != SMLA_Q8_E4M3 && c->format != SMLA_Q8_INT8) return SMLA_ERR_UNSUPPORTED;
  if (c->h_kv < 1 || c->h_kv > 65535 || (int64_t)c->h_kv * c->head_dim * smla::kBlk > 0x7FFFFFFF)
    return SMLA_ERR_INVALID_ARGUMENT;
  if (!c->k_cache || !c->v_cache || !c->k_scale || !c->v_scale) return SMLA_ERR_INVALID_ARGUMENT;
  const int64_t dense = (int64_t)c->h_kv * c->head_dim * smla::kBlk;
  if (c->num_blocks < 1 || c->num_blocks > 0x7FFFFFFF / smla::kBlk) return SMLA_ERR_INVALID_ARGUMENT;
  if (c->k_block_stride < dense || c->v_block_stride < dense || c->k_block_stride % 16 || c->v_block_stride % 16 ||
      c->k_block_stride >= ((int64_t)1 << 40) || c->v_block_stride >= ((int64_t)1 << 40))
    return SMLA_ERR_INVALID_ARGUMENT;
  if (c->k_scale_stride < c->h_kv || c->v_scale_stride < c->h_kv || c->k_scale_stride > kMost ||
      c->v_scale_stride > kMost)
    return SMLA_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return SMLA_ERR_INVALID_ARGUMENT;
  return SMLA_OK;
}

// A cap whose inverse and whose products with scores stay well inside fp32.
bool good_cap(float x) { return x >= 0x1p-60f && x <= 0x1p60f; }

bool good_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s <= kMost / 0x10000; }

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// The paged cache as (d, token, head, block), one (head, block) tile a copy.
int tile_map(CUtensorMap* map, void* base, const smla_q8_cache* c, int64_t block_stride) {
  const EncodeFn enc = encoder();
  if (!enc) return smla::cuda_failure(cudaErrorNotSupported);
  const cuuint64_t d = (cuuint64_t)c->head_dim;
  const cuuint64_t size[4] = {d, smla::kBlk, (cuuint64_t)c->h_kv, (cuuint64_t)c->num_blocks};
  const cuuint64_t stride[3] = {d, d * smla::kBlk, (cuuint64_t)block_stride};
  const cuuint32_t box[4] = {(cuuint32_t)d, smla::kBlk, 1, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, size, stride, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SMLA_OK : smla::cuda_failure(cudaErrorInvalidValue);
}

constexpr int kMaxDevices = 64;

// SM count of a device, and whether it is sm_100; asked of the runtime once.
int device_facts(int device, int* sms, bool* sm100) {
  static std::atomic<int> known[kMaxDevices];         // 0: not asked; else SMs * 2 + sm_100
  if (device < 0 || device >= kMaxDevices) return SMLA_ERR_UNSUPPORTED;
  int f = known[device].load(std::memory_order_relaxed);
  if (f == 0) {
    int n = 0, major = 0, minor = 0;
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device);
    if (e != cudaSuccess) return smla::cuda_failure(e);
    f = (n > 0 ? n : 1) * 2 + (major == 10 && minor == 0 ? 1 : 0);
    known[device].store(f, std::memory_order_relaxed);
  }
  *sms = f >> 1;
  *sm100 = f & 1;
  return SMLA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t cta_o_off, lse_off, cta_lse_off, meta_off, total;
};

Layout workspace(int head_dim, int ctas) {
  const size_t warps = (size_t)ctas * smla::kQ8DecodeWarps, rows = 2 * smla::kQ8PartRows;
  Layout l;
  l.cta_o_off = align256(rows * warps * (size_t)head_dim * sizeof(float));
  l.lse_off = l.cta_o_off + align256(rows * (size_t)ctas * (size_t)head_dim * sizeof(float));
  l.cta_lse_off = l.lse_off + align256(rows * warps * sizeof(float));
  l.meta_off = l.cta_lse_off + align256(rows * (size_t)ctas * sizeof(float));
  l.total = l.meta_off + align256((size_t)ctas * 8 * sizeof(int32_t));
  return l;
}

}  // namespace

namespace smla {

cudaError_t raise_shared_limit(SharedLimit& done, const void* kernel, int bytes) {
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  void* ctx = current_context();
  std::atomic<void*>& known = done.done[dev & 63];
  if (dev < 64 && ctx != nullptr && known.load(std::memory_order_acquire) == ctx) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) known.store(ctx != nullptr ? ctx : current_context(), std::memory_order_release);
  return e;
}

}  // namespace smla

extern "C" {

int smla_quantize_kv_blocks(const void* k, const void* v, int64_t k_token_stride, int64_t k_head_stride,
                            int64_t v_token_stride, int64_t v_head_stride, int64_t total_new,
                            const smla_q8_cache* cache, const int32_t* block_table, int max_blocks, int batch,
                            const int32_t* cache_seqlens, const int32_t* new_seqlens, const int32_t* cu_new,
                            uint32_t* status, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (batch < 0 || max_blocks < 1 || total_new < 0 || total_new > 0x7FFFFFFF || batch > (1 << 28))
    return SMLA_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_new == 0) return SMLA_OK;
  if (!k || !v || !block_table || !cache_seqlens || !new_seqlens || !cu_new) return SMLA_ERR_INVALID_ARGUMENT;
  if (!aligned(k, 16) || !aligned(v, 16) || !good_stride(k_token_stride) || !good_stride(k_head_stride) ||
      !good_stride(v_token_stride) || !good_stride(v_head_stride))
    return SMLA_ERR_INVALID_ARGUMENT;
  smla::Q8WriteParams p;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_token_stride = k_token_stride;
  p.k_head_stride = k_head_stride;
  p.v_token_stride = v_token_stride;
  p.v_head_stride = v_head_stride;
  p.k_cache = static_cast<uint8_t*>(cache->k_cache);
  p.v_cache = static_cast<uint8_t*>(cache->v_cache);
  p.k_block_bytes = cache->k_block_stride;
  p.v_block_bytes = cache->v_block_stride;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.k_scale_stride = cache->k_scale_stride;
  p.v_scale_stride = cache->v_scale_stride;
  p.num_blocks = cache->num_blocks;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.new_seqlens = new_seqlens;
  p.cu = cu_new;
  p.max_blocks = max_blocks;
  p.batch = batch;
  p.total = (int)total_new;
  p.h_kv = cache->h_kv;
  p.status = status;
  const cudaError_t e =
      smla::launch_q8_write(p, cache->head_dim, cache->format == SMLA_Q8_INT8, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SMLA_OK : smla::cuda_failure(e);
}

size_t smla_gqa_workspace_bytes(int head_dim, int device) {
  int sms = 0;
  bool sm100 = false;
  if ((head_dim != 64 && head_dim != 128) || device_facts(device, &sms, &sm100)) return 0;
  return workspace(head_dim, sms).total;
}

int smla_gqa_attention_with_kvcache(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t total_q,
                                    int h_q, const smla_q8_cache* cache, const int32_t* block_table, int max_blocks,
                                    int batch, const int32_t* cache_seqlens, const int32_t* cu_seqlens_q, int s_q,
                                    int max_seqlen_q, int causal, float softmax_scale, float softcap,
                                    const float* alibi_slopes, const int32_t* prefix_lens, const int32_t* doc_bounds,
                                    void* o, float* lse, void* workspace_ptr, size_t workspace_bytes,
                                    uint32_t* status, void* stream) {
  if (int rc = check_cache(cache)) return rc;
  if (h_q < 1 || h_q >= (1 << 20) || h_q % cache->h_kv != 0 || batch < 0 || batch > (1 << 28) || max_blocks < 1)
    return SMLA_ERR_INVALID_ARGUMENT;
  if (total_q < 0 || total_q > 0x7FFFFFFF || total_q * h_q > 0x7FFFFFFF || (causal != 0 && causal != 1) ||
      max_seqlen_q < 0)
    return SMLA_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens_q && (s_q < 0 || (int64_t)batch * s_q != total_q)) return SMLA_ERR_INVALID_ARGUMENT;
  if (softcap != 0.f && !good_cap(softcap)) return SMLA_ERR_INVALID_ARGUMENT;
  if (softmax_scale > 0.f && !std::isnormal(softmax_scale)) return SMLA_ERR_INVALID_ARGUMENT;
  if (prefix_lens && !causal) return SMLA_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_q == 0) return SMLA_OK;
  if (!q || !block_table || !cache_seqlens || !o || !lse || !workspace_ptr) return SMLA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace_ptr, 256) || !aligned(doc_bounds, 8) ||
      !good_stride(q_token_stride) || !good_stride(q_head_stride))
    return SMLA_ERR_INVALID_ARGUMENT;
  int dev = 0, sms = 0;
  bool sm100 = false;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return smla::cuda_failure(e);
  if (int rc = device_facts(dev, &sms, &sm100)) return rc;
  if (!sm100) return SMLA_ERR_UNSUPPORTED;
  const Layout wl = workspace(cache->head_dim, sms);
  if (workspace_bytes < wl.total) return SMLA_ERR_INVALID_ARGUMENT;

  smla::Q8Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.k_scale_stride = cache->k_scale_stride;
  p.v_scale_stride = cache->v_scale_stride;
  p.k_cache = static_cast<const uint8_t*>(cache->k_cache);
  p.v_cache = static_cast<const uint8_t*>(cache->v_cache);
  p.k_block_bytes = cache->k_block_stride;
  p.v_block_bytes = cache->v_block_stride;
  p.num_blocks = cache->num_blocks;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.cu_q = cu_seqlens_q;
  p.slopes = alibi_slopes;
  p.prefix = prefix_lens;
  p.docs = doc_bounds;
  p.max_blocks = max_blocks;
  p.batch = batch;
  p.s_q = s_q;
  p.total_q = (int)total_q;
  p.h_q = h_q;
  p.h_kv = cache->h_kv;
  p.group = h_q / cache->h_kv;
  p.inv_group = 1.0f / (float)p.group;
  p.d = cache->head_dim;
  p.causal = causal;
  p.scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)cache->head_dim);
  p.cap = softcap;
  p.cap_log2 = softcap * smla::kLog2e;
  p.inv_cap_log2 = softcap > 0.f ? 1.0f / p.cap_log2 : 0.f;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.status = status;
  const bool int8 = cache->format == SMLA_Q8_INT8;
  uint8_t* ws = static_cast<uint8_t*>(workspace_ptr);
  smla::Q8Scratch scratch;
  scratch.o = reinterpret_cast<float*>(ws);
  scratch.cta_o = reinterpret_cast<float*>(ws + wl.cta_o_off);
  scratch.lse = reinterpret_cast<float*>(ws + wl.lse_off);
  scratch.cta_lse = reinterpret_cast<float*>(ws + wl.cta_lse_off);
  scratch.meta = reinterpret_cast<int32_t*>(ws + wl.meta_off);
  const int rows = (int)(std::min<int64_t>(max_seqlen_q, total_q) * p.group);   // below 2^31, as total_q * h_q is
  if (!smla::q8_decode_pays(batch, cache->h_kv, p.group, total_q, max_seqlen_q, doc_bounds != nullptr, sms)) {
    const cudaError_t e = smla::launch_q8_prefill(p, int8, rows, scratch, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SMLA_OK : smla::cuda_failure(e);
  }
  CUtensorMap k_map, v_map;
  if (int rc = tile_map(&k_map, cache->k_cache, cache, cache->k_block_stride)) return rc;
  if (int rc = tile_map(&v_map, cache->v_cache, cache, cache->v_block_stride)) return rc;
  const cudaError_t e = smla::launch_q8_decode(p, int8, rows, k_map, v_map, scratch, sms,
                                               static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SMLA_OK : smla::cuda_failure(e);
}

}  // extern "C"
