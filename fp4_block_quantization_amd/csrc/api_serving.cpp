// C ABI of the token-serving operators: argument validation (before any HIP call) and
// kernel dispatch.  See include/fos.h for the contract of every entry point.
#include "../../include/fos.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "kernels.hpp"
#include "serving.hpp"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;   // work-items of one launch
constexpr int kMinPage = 16, kMaxPage = 4096;
constexpr int kMaxHeadDim = 256;
constexpr int kMaxHeads = 65536;   // keeps the index arithmetic of the cache kernels in range
constexpr int64_t kMaxTokens = (int64_t)1 << 30;   // of one sequence
constexpr int64_t kMaxBatchTokens = (int64_t)1 << 38;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fos_status status_of(hipError_t e) { return e == hipSuccess ? FOS_OK : FOS_E_HIP; }

fos_status check_wlinear(const fos::WLinearArgs& a, int out_dtype) {
  const int64_t block = a.mx ? 32 : 16;
  if (out_dtype != FOS_OUT_F32 && out_dtype != FOS_OUT_BF16) return FOS_E_FLAGS;
  if (a.M < 0 || a.N < 1 || a.K < block || a.K % block || a.M >= kMaxDim || a.N >= kMaxDim ||
      a.K >= kMaxDim)
    return FOS_E_SHAPE;
  if (a.K > kMaxElems / a.N || (a.M > 0 && (a.N > kMaxElems / a.M || a.K > kMaxElems / a.M)))
    return FOS_E_SHAPE;
  if (a.x_stride < 0 || (a.M > 1 && (a.x_stride < a.K || a.x_stride > kMaxElems / a.M)))
    return FOS_E_SHAPE;
  if (a.M == 0) return FOS_OK;
  if (fos::wlinear_threads(a) > kMaxThreads) return FOS_E_SHAPE;
  if (!a.x || !a.wd || !a.ws || !a.y || (!a.mx && !a.wt)) return FOS_E_NULL;
  if (!aligned(a.x, 16) || (a.M > 1 && a.x_stride % 8) || !aligned(a.wd, 16) ||
      !aligned(a.ws, 4) || (!a.mx && !aligned(a.wt, 4)) || (a.bias && !aligned(a.bias, 2)) ||
      !aligned(a.y, out_dtype == FOS_OUT_F32 ? 4 : 2))
    return FOS_E_ALIGN;
  return FOS_OK;
}

fos_status run_wlinear(const void* x, int64_t x_stride, const uint8_t* wd, const uint8_t* ws,
                       const float* wt, const void* bias, int64_t M, int64_t N, int64_t K,
                       int out_dtype, void* y, bool mx, void* stream) {
  fos::WLinearArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.wd = wd;
  a.ws = ws;
  a.wt = wt;
  a.bias = static_cast<const uint16_t*>(bias);
  a.y = y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.mx = mx;
  a.f32_out = out_dtype == FOS_OUT_F32;
  const fos_status st = check_wlinear(a, out_dtype);
  if (st != FOS_OK || M == 0) return st;
  return status_of(fos::launch_wlinear(a, static_cast<hipStream_t>(stream)));
}

fos_status check_cache(const fos_kv_cache* c) {
  if (!c) return FOS_E_NULL;
  if (c->struct_size != sizeof(fos_kv_cache) || c->reserved != 0 ||
      (c->format != FOS_KV_BF16 && c->format != FOS_KV_NVFP4))
    return FOS_E_FLAGS;
  if (c->num_pages < 0 || c->num_pages >= kMaxDim || c->page_size < kMinPage ||
      c->page_size > kMaxPage || c->page_size % 16 || c->num_kv_heads < 1 ||
      c->num_kv_heads > kMaxHeads || c->head_dim < 32 ||
      c->head_dim > kMaxHeadDim || c->head_dim % 32)
    return FOS_E_SHAPE;
  const int64_t row = (int64_t)c->page_size * c->head_dim;   // at most 2^20
  if (c->num_kv_heads > kMaxElems / row ||
      (c->num_pages > 0 && c->num_kv_heads * row > kMaxElems / c->num_pages))
    return FOS_E_SHAPE;
  if (c->num_pages == 0) return FOS_OK;
  if (!c->k_data || !c->v_data) return FOS_E_NULL;
  if (!aligned(c->k_data, 16) || !aligned(c->v_data, 16)) return FOS_E_ALIGN;
  if (c->format == FOS_KV_NVFP4) {
    if (!c->k_scales || !c->v_scales || !c->k_tensor_scale || !c->v_tensor_scale)
      return FOS_E_NULL;
    if (!aligned(c->k_scales, 16) || !aligned(c->v_scales, 16) ||
        !aligned(c->k_tensor_scale, 4) || !aligned(c->v_tensor_scale, 4))
      return FOS_E_ALIGN;
  }
  return FOS_OK;
}

fos::KVCacheArgs cache_args(const fos_kv_cache* c) {
  fos::KVCacheArgs a;
  a.nvfp4 = c->format == FOS_KV_NVFP4;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.heads = c->num_kv_heads;
  a.dim = c->head_dim;
  a.k = static_cast<uint8_t*>(c->k_data);
  a.v = static_cast<uint8_t*>(c->v_data);
  a.ks = c->k_scales;
  a.vs = c->v_scales;
  a.kt = c->k_tensor_scale;
  a.vt = c->v_tensor_scale;
  return a;
}

// Rows of new tokens: [token][kv head][dim] with a token stride.
fos_status check_rows(const fos_kv_cache* c, const int64_t* slots, int64_t T, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride) {
  const fos_status st = check_cache(c);
  if (st != FOS_OK) return st;
  const int64_t width = (int64_t)c->num_kv_heads * c->head_dim;
  if (T < 0 || T >= kMaxDim || k_stride < 0 || v_stride < 0) return FOS_E_SHAPE;
  if (T > 0 && (width > kMaxElems / T || k_stride > kMaxElems / T || v_stride > kMaxElems / T))
    return FOS_E_SHAPE;
  // the finest kernel takes one thread per 8 values
  if ((T * width / 8 + 255) / 256 > fos::kMaxGrid) return FOS_E_SHAPE;
  if (T > 1 && (k_stride < width || v_stride < width)) return FOS_E_SHAPE;
  if (T == 0) return FOS_OK;
  if (!slots || !k || !v) return FOS_E_NULL;
  if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16) ||
      (T > 1 && (k_stride % 8 || v_stride % 8)))
    return FOS_E_ALIGN;
  return FOS_OK;
}

fos::KVRowsArgs rows_args(const fos_kv_cache* c, const int64_t* slots, int64_t T, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride) {
  fos::KVRowsArgs a;
  a.c = cache_args(c);
  a.slots = slots;
  a.T = T;
  a.k = static_cast<uint16_t*>(const_cast<void*>(k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(v));
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.four_over_six = true;
  return a;
}

}  // namespace

extern "C" {

fos_status fos_wlinear_fwd(const void* x_bf16, int64_t x_stride, const uint8_t* w_data,
                           const uint8_t* w_scales, const float* w_tensor_scale,
                           const void* bias_bf16, int64_t M, int64_t N, int64_t K, int out_dtype,
                           void* y, void* stream) {
  return run_wlinear(x_bf16, x_stride, w_data, w_scales, w_tensor_scale, bias_bf16, M, N, K,
                     out_dtype, y, false, stream);
}

fos_status fos_mx_wlinear_fwd(const void* x_bf16, int64_t x_stride, const uint8_t* w_data,
                              const uint8_t* w_scales, const void* bias_bf16, int64_t M,
                              int64_t N, int64_t K, int out_dtype, void* y, void* stream) {
  return run_wlinear(x_bf16, x_stride, w_data, w_scales, nullptr, bias_bf16, M, N, K, out_dtype,
                     y, true, stream);
}

fos_status fos_kv_append(const fos_kv_cache* cache, int rule, const void* k_bf16,
                         int64_t k_stride, const void* v_bf16, int64_t v_stride,
                         const int64_t* slots, int64_t num_tokens, void* stream) {
  const fos_status st = check_rows(cache, slots, num_tokens, k_bf16, k_stride, v_bf16, v_stride);
  if (st != FOS_OK) return st;
  if (rule != FOS_RULE_4OVER6 && rule != FOS_RULE_6ONLY) return FOS_E_FLAGS;
  if (num_tokens == 0 || cache->num_pages == 0) return FOS_OK;
  fos::KVRowsArgs a = rows_args(cache, slots, num_tokens, k_bf16, k_stride, v_bf16, v_stride);
  a.four_over_six = rule == FOS_RULE_4OVER6;
  return status_of(fos::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

fos_status fos_kv_gather(const fos_kv_cache* cache, const int64_t* slots, int64_t num_tokens,
                         void* k_bf16, int64_t k_stride, void* v_bf16, int64_t v_stride,
                         void* stream) {
  const fos_status st = check_rows(cache, slots, num_tokens, k_bf16, k_stride, v_bf16, v_stride);
  if (st != FOS_OK || num_tokens == 0) return st;
  return status_of(fos::launch_kv_gather(
      rows_args(cache, slots, num_tokens, k_bf16, k_stride, v_bf16, v_stride),
      static_cast<hipStream_t>(stream)));
}

size_t fos_paged_decode_workspace_bytes(int64_t num_seqs, int64_t num_q_heads,
                                        int64_t num_kv_heads, int64_t head_dim) {
  if (num_seqs < 0 || num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads ||
      head_dim < 1 || head_dim > kMaxHeadDim || num_q_heads >= kMaxDim || num_seqs >= kMaxDim ||
      num_seqs * num_q_heads >= kMaxDim || !fos::decode_heads_ok(num_q_heads, num_kv_heads))
    return 0;
  return fos::decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim);
}

size_t fos_paged_decode_counter_bytes(void) { return fos::kCounterBytes; }

fos_status fos_paged_decode(const fos_kv_cache* cache, const void* q_bf16, int64_t q_stride,
                            int64_t num_seqs, int64_t num_q_heads, const int32_t* block_table,
                            int64_t table_stride, int64_t pages_per_seq, const int32_t* seq_lens,
                            float softmax_scale, int64_t window, void* out_bf16, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream) {
  fos_status st = check_cache(cache);
  if (st != FOS_OK) return st;
  if (num_seqs < 0 || num_q_heads < 1 || num_q_heads % cache->num_kv_heads ||
      num_seqs >= kMaxDim || num_q_heads >= kMaxDim || num_seqs * num_q_heads >= kMaxDim ||
      pages_per_seq < 0 || pages_per_seq >= kMaxDim ||
      pages_per_seq * cache->page_size > kMaxTokens || q_stride < 0 || table_stride < 0)
    return FOS_E_SHAPE;
  const int64_t width = num_q_heads * cache->head_dim;
  if (num_seqs > 1 && (q_stride < width || table_stride < pages_per_seq ||
                       q_stride > kMaxElems / num_seqs || table_stride > kMaxElems / num_seqs))
    return FOS_E_SHAPE;
  // the device counts steps of 256 tokens of all sequences in 32 bits
  const int64_t cap = pages_per_seq * cache->page_size;
  if (num_seqs > 0 && cap > kMaxBatchTokens / num_seqs) return FOS_E_SHAPE;
  if (!fos::decode_heads_ok(num_q_heads, cache->num_kv_heads)) return FOS_E_SHAPE;
  if (window < 0 || !std::isfinite(softmax_scale)) return FOS_E_FLAGS;
  if (num_seqs == 0) return FOS_OK;
  if (!q_bf16 || !seq_lens || !out_bf16 || (pages_per_seq > 0 && !block_table)) return FOS_E_NULL;
  if (!aligned(q_bf16, 16) || (num_seqs > 1 && q_stride % 8) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(out_bf16, 16) || !aligned(lse, 4))
    return FOS_E_ALIGN;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < fos_paged_decode_workspace_bytes(num_seqs, num_q_heads,
                                                         cache->num_kv_heads, cache->head_dim))
    return FOS_E_WORKSPACE;
  fos::DecodeArgs a;
  a.c = cache_args(cache);
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.q_stride = q_stride;
  a.B = (int)num_seqs;
  a.Hq = (int)num_q_heads;
  a.G = (int)(num_q_heads / cache->num_kv_heads);
  a.table = block_table;
  a.table_stride = table_stride;
  // An empty cache holds no page: nothing is visible.  Its pointers may be null, and the
  // kernel of a bf16 cache, unlike that of an NVFP4 one, reads none before it sees a token.
  a.pages_per_seq = cache->num_pages > 0 ? (int)pages_per_seq : 0;
  if (cache->num_pages == 0) a.c.nvfp4 = false;
  a.lens = seq_lens;
  a.scale = softmax_scale;
  a.window = window;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.lse = lse;
  a.ws = workspace;
  return status_of(fos::launch_paged_decode(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
