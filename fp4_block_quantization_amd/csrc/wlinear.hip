// Weight-only quantized linear layer: bf16 activations times a 4-bit weight record,
//   y[m][n] = t * sum_k x[m][k] E(w[n][k]) D(s[n][k / block]) + bias[n].
// Products are exact in fp32 (8 x 2 significant bits), the sum over a block is scaled
// by its block scale, and every sum is fp32; y is rounded once.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsX = 8;   // activation rows per pass over a weight row

// One wave per weight row, one scale block per lane and step.
template <bool kMX>
__global__ __launch_bounds__(kThreads) void wlinear_kernel(WLinearArgs a) {
  constexpr int kBlock = kMX ? 32 : 16;
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const int64_t nblk = a.K / kBlock;
  const float t = kMX ? 1.0f : a.wt[0];
  for (int64_t m0 = 0; m0 < a.M; m0 += kRowsX) {
    const int rows = (int)min((int64_t)kRowsX, a.M - m0);
    float acc[kRowsX];
#pragma unroll
    for (int m = 0; m < kRowsX; ++m) acc[m] = 0.0f;
    for (int64_t b = lane; b < nblk; b += 64) {
      const uint32_t sb = a.ws[n * nblk + b];
      const float d = kMX ? ldexpf(1.0f, (int)sb - 127) : e4m3_decode(sb & 0x7f);
      float part[kRowsX];
#pragma unroll
      for (int m = 0; m < kRowsX; ++m) part[m] = 0.0f;
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(a.wd + n * (a.K / 2) + b * (kBlock / 2));
#pragma unroll
      for (int j = 0; j < kBlock / 8; ++j) {
        const uint32_t w = wp[j];
        const f32x2 e[4] = {cvt_pk_f32_fp4<0>(w), cvt_pk_f32_fp4<1>(w), cvt_pk_f32_fp4<2>(w),
                            cvt_pk_f32_fp4<3>(w)};
#pragma unroll
        for (int m = 0; m < kRowsX; ++m) {
          if (m >= rows) break;
          const uint4 x = *reinterpret_cast<const uint4*>(a.x + (m0 + m) * a.x_stride + b * kBlock + 8 * j);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            part[m] = __builtin_fmaf(bf16_lo(xw[i]), e[i].x, part[m]);
            part[m] = __builtin_fmaf(bf16_hi(xw[i]), e[i].y, part[m]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kRowsX; ++m) acc[m] = __builtin_fmaf(part[m], d, acc[m]);
    }
#pragma unroll
    for (int m = 0; m < kRowsX; ++m) {
      if (m >= rows) break;
      float v = acc[m];
      for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
      if (lane == 0) {
        v *= t;
        if (a.bias) v += bf16_lo(a.bias[n]);
        const int64_t o = (m0 + m) * a.N + n;
        if (a.f32_out) static_cast<float*>(a.y)[o] = v;
        else static_cast<uint16_t*>(a.y)[o] = (uint16_t)pack_bf16x2(v, v);
      }
    }
  }
}

}  // namespace

hipError_t launch_wlinear(const WLinearArgs& a, hipStream_t s) {
  const uint32_t grid = (uint32_t)((a.N + 3) / 4);
  if (a.mx) wlinear_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else wlinear_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fos
