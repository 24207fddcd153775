// Attention of one new token per sequence over a paged key-value cache.  For sequence b
// and query head h (kv head h / G), over the visible tokens j (below the length, inside
// the window, in a page that the cache holds):
//   s_j = scale * q . k_j,   lse = log sum exp s_j,   out = sum exp(s_j - lse) v_j,
// in one pass over K and V with the running maximum m and sum l of the softmax:
//   m' = max(m, s),  l' = l exp(m - m') + exp(s - m'),  o' = o exp(m - m') + exp(s - m') v.
// Statistics, products and sums are fp32; out is rounded once.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = 4;      // values of a row per lane (dim <= 256)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

template <bool kNVFP4>
__device__ __forceinline__ float cache_value(const uint8_t* data, const uint8_t* scales,
                                             int64_t row, int dim, int d) {
  if (!kNVFP4) return bf16_lo(reinterpret_cast<const uint16_t*>(data)[row * dim + d]);
  const uint32_t byte = data[row * (dim / 2) + d / 2];
  const f32x2 e = cvt_pk_f32_fp4<0>(byte);
  return (d & 1 ? e.y : e.x) * e4m3_decode(scales[row * (dim / 16) + d / 16]);
}

// One workgroup per (sequence, query head); wave w takes tokens w, w + 4, ...
template <bool kNVFP4>
__global__ __launch_bounds__(kThreads) void paged_decode_kernel(DecodeArgs a) {
  __shared__ float sm[kWaves], sl[kWaves], so[kWaves][256];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / a.G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, dim = a.c.dim;
  const int64_t cap = (int64_t)a.pages_per_seq * a.c.page_size;
  const int64_t L = min((int64_t)a.lens[b], cap);
  const int64_t first = a.window > 0 ? max((int64_t)0, (int64_t)a.lens[b] - a.window) : 0;
  const float kt = kNVFP4 ? a.c.kt[0] : 1.0f, vt = kNVFP4 ? a.c.vt[0] : 1.0f;
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = lane + 64 * i;
    q[i] = d < dim ? bf16_lo(a.q[b * a.q_stride + (int64_t)h * dim + d]) : 0.0f;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = first + wave; j < L; j += kWaves) {
    const int64_t pj = j / a.c.page_size;
    const int page = a.table[b * a.table_stride + pj];
    if (page < 0 || page >= a.c.num_pages) continue;
    const int64_t row = ((int64_t)page * a.c.heads + hk) * a.c.page_size + (j - pj * a.c.page_size);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane + 64 * i;
      if (d < dim) s = __builtin_fmaf(q[i], cache_value<kNVFP4>(a.c.k, a.c.ks, row, dim, d), s);
    }
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    s *= a.scale * kt * kLog2e;
    const float m2 = fmaxf(m, s);
    const float f = exp2f(m - m2), p = exp2f(s - m2);
    m = m2;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane + 64 * i;
      if (d < dim) o[i] = o[i] * f + p * cache_value<kNVFP4>(a.c.v, a.c.vs, row, dim, d);
    }
  }
  if (lane == 0) { sm[wave] = m; sl[wave] = l; }
#pragma unroll
  for (int i = 0; i < kPer; ++i) so[wave][lane + 64 * i] = o[i];
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, sm[w]);
  float ll = 0.0f, oo = 0.0f;
  for (int w = 0; w < kWaves; ++w) {
    if (sm[w] == -INFINITY) continue;
    const float f = exp2f(sm[w] - mm);
    ll += sl[w] * f;
    oo += so[w][threadIdx.x] * f;
  }
  if ((int)threadIdx.x < dim) {
    const float r = ll > 0.0f ? oo / ll * vt : 0.0f;
    a.out[((int64_t)b * a.Hq + h) * dim + threadIdx.x] = (uint16_t)pack_bf16x2(r, r);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(int64_t)b * a.Hq + h] = ll > 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
}

}  // namespace

size_t decode_workspace_bytes(int64_t, int64_t, int64_t, int64_t) { return 16; }

hipError_t launch_paged_decode(const DecodeArgs& a, hipStream_t s) {
  const uint32_t grid = (uint32_t)a.B * (uint32_t)a.Hq;
  if (a.c.nvfp4) paged_decode_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else paged_decode_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fos
