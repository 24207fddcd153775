// Paged key-value cache: append rows of new tokens to their slots and read slots back.
//
// The cache is [page][kv head][token of the page][value], so a page holds each head's
// tokens in one run; an NVFP4 page of a head is an NVFP4 record [page_size][dim] (16
// values of a row per E4M3 block scale, static fp32 tensor scales for all of K and all
// of V).  Slot = page * page_size + token of the page; a slot outside the cache is
// skipped (append) or read as zeros (gather).
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;

// Row (slot, head) of the cache, or -1.
__device__ __forceinline__ int64_t cache_row(const KVCacheArgs& c, int64_t slot, int head) {
  if (slot < 0 || slot >= c.num_pages * c.page_size) return -1;
  const int64_t page = slot / c.page_size;
  return (page * c.heads + head) * c.page_size + (slot - page * c.page_size);
}

// One thread per 16 values of one row of K (blockIdx.y 0) or V (1).
template <bool k46>
__global__ __launch_bounds__(kThreads) void append_nvfp4_kernel(KVRowsArgs a) {
  __shared__ float2 tab[kScaleTableSize];
  const bool is_v = blockIdx.y != 0;
  const float t = is_v ? a.c.vt[0] : a.c.kt[0];
  build_scale_table(tab, t);
  const int nb = a.c.dim / 16, per = nb * a.c.heads;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.T * per) return;
  const int64_t tok = i / per;
  const int r = (int)(i - tok * per);
  const int64_t row = cache_row(a.c, a.slots[tok], r / nb);
  if (row < 0) return;
  const uint16_t* src = (is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) + 16 * r;
  const uint4 w0 = reinterpret_cast<const uint4*>(src)[0];
  const uint4 w1 = reinterpret_cast<const uint4*>(src)[1];
  float v[16];
  unpack16(w0, w1, v);
  const uint32_t none[16] = {};
  const Cand c = quantize_block<k46, false>(v, tab, tab[128].x, tab[128].y, none);
  const int64_t blk = row * nb + r % nb;
  *reinterpret_cast<uint2*>((is_v ? a.c.v : a.c.k) + 8 * blk) = make_uint2(c.lo, c.hi);
  (is_v ? a.c.vs : a.c.ks)[blk] = (uint8_t)c.s;
}

// One thread per 8 values.
__global__ __launch_bounds__(kThreads) void append_bf16_kernel(KVRowsArgs a) {
  const bool is_v = blockIdx.y != 0;
  const int nb = a.c.dim / 8, per = nb * a.c.heads;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.T * per) return;
  const int64_t tok = i / per;
  const int r = (int)(i - tok * per);
  const int64_t row = cache_row(a.c, a.slots[tok], r / nb);
  if (row < 0) return;
  const uint16_t* src = (is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) + 8 * r;
  reinterpret_cast<uint4*>(is_v ? a.c.v : a.c.k)[row * nb + r % nb] =
      *reinterpret_cast<const uint4*>(src);
}

// One thread per 8 values.
template <bool kNVFP4>
__global__ __launch_bounds__(kThreads) void gather_kernel(KVRowsArgs a) {
  const bool is_v = blockIdx.y != 0;
  const int nb = a.c.dim / 8, per = nb * a.c.heads;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.T * per) return;
  const int64_t tok = i / per;
  const int r = (int)(i - tok * per);
  const int64_t row = cache_row(a.c, a.slots[tok], r / nb);
  uint4 o = make_uint4(0, 0, 0, 0);
  if (row >= 0) {
    const int64_t at = row * nb + r % nb;
    if (kNVFP4) {
      const uint32_t q = reinterpret_cast<const uint32_t*>(is_v ? a.c.v : a.c.k)[at];
      const float d = e4m3_decode((is_v ? a.c.vs : a.c.ks)[at >> 1]) * (is_v ? a.c.vt[0] : a.c.kt[0]);
      const f32x2 e0 = cvt_pk_f32_fp4<0>(q), e1 = cvt_pk_f32_fp4<1>(q);
      const f32x2 e2 = cvt_pk_f32_fp4<2>(q), e3 = cvt_pk_f32_fp4<3>(q);
      o = make_uint4(pack_bf16x2(e0.x * d, e0.y * d), pack_bf16x2(e1.x * d, e1.y * d),
                     pack_bf16x2(e2.x * d, e2.y * d), pack_bf16x2(e3.x * d, e3.y * d));
    } else {
      o = reinterpret_cast<const uint4*>(is_v ? a.c.v : a.c.k)[at];
    }
  }
  uint16_t* dst = (is_v ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) + 8 * r;
  *reinterpret_cast<uint4*>(dst) = o;
}

dim3 rows_grid(const KVRowsArgs& a, int values) {
  const int64_t n = a.T * a.c.heads * (a.c.dim / values);
  return dim3((uint32_t)((n + kThreads - 1) / kThreads), 2);
}

}  // namespace

hipError_t launch_kv_append(const KVRowsArgs& a, hipStream_t s) {
  if (!a.c.nvfp4) append_bf16_kernel<<<rows_grid(a, 8), kThreads, 0, s>>>(a);
  else if (a.four_over_six) append_nvfp4_kernel<true><<<rows_grid(a, 16), kThreads, 0, s>>>(a);
  else append_nvfp4_kernel<false><<<rows_grid(a, 16), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_gather(const KVRowsArgs& a, hipStream_t s) {
  if (a.c.nvfp4) gather_kernel<true><<<rows_grid(a, 8), kThreads, 0, s>>>(a);
  else gather_kernel<false><<<rows_grid(a, 8), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fos
