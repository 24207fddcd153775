// Epilogue of the GEMM kernels' tiles with bias, activation, gate and residual.
//
// A wave's accumulators hold one column and 16 rows of each 32x32 tile a lane; y is written,
// and the residual read, fastest where a lane has neighbouring columns.  So each strip of 32
// rows goes through the wave's own LDS as fp32 and comes back four columns to a lane: whole
// 128- or 256-byte runs of a row a wave instruction, and one short loop that knows the
// activation instead of 256 unrolled values that each do.
#pragma once

#include "activation.hpp"
#include "gemm_common.hpp"

namespace fos {
namespace gemm {

// What a GEMM kernel does with its sums: kPlain stores them, kFused applies the epilogue,
// kGated too, with gate and other projection in neighbouring 32-column tiles.
enum { kPlain, kFused, kGated };

// Floats between rows of a strip: a multiple of 4 (16-byte reads) with 4 rows apart half the
// banks (the two lane halves of a write are 4 rows apart).
template <int TJ>
constexpr int kStripStride = 32 * TJ + 8;
template <int TJ>
constexpr int kStripBytes = 32 * kStripStride<TJ> * 4;   // of each wave

// Weight row behind row r (0 .. 64 TJ - 1) of a gated tile, without the tile's first column:
// rows come in groups of 32, gate and other projection in turn; `up` says which.
__device__ __forceinline__ int gated_row(int r, bool& up) {
  up = (r >> 5) & 1;
  return ((r >> 6) << 5) | (r & 31);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Four columns from `n` of a row; those past N (of which `left` remain) are not touched.
__device__ __forceinline__ f32x4 load_bf16x4(const uint16_t* p, bool wide, int left) {
  if (wide) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
  }
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) v[i] = bf16_lo(p[i]);
  return v;
}
__device__ __forceinline__ void store_bf16x4(uint16_t* p, f32x4 v, bool wide, int left) {
  const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (wide) {
    *reinterpret_cast<u32x2*>(p) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) p[i] = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
}
__device__ __forceinline__ void store_f32x4(float* p, f32x4 v, bool wide, int left) {
  if (wide) {
    *reinterpret_cast<f32x4*>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) p[i] = v[i];
}

// One strip: rows m0 .. m0 + 31, the wave's columns from n0 (of y).
template <int TJ, bool kGate, int kAct>
__device__ __forceinline__ void fused_strip(const EpilogueArgs& e, void* y, const float* strip,
                                            int M, int N, int m0, int n0, int lane,
                                            f32x4 bias, f32x4 bias_up) {
  constexpr int kS = kStripStride<TJ>;
  constexpr int kCols = kGate ? 16 * TJ : 32 * TJ, kAcross = kCols / 4, kRows = 64 / kAcross;
  const int c = 4 * (lane % kAcross), r0 = lane / kAcross;
  const int col = kGate ? 64 * (c >> 5) + (c & 31) : c;
  const int n = n0 + c, left = N - n;
  if (left <= 0) return;
  const bool wide = e.wide && left >= 4;
#pragma unroll 4
  for (int i = 0; i < 32 / kRows; ++i) {
    const int r = i * kRows + r0;
    const int64_t m = m0 + r;
    f32x4 z = *reinterpret_cast<const f32x4*>(strip + r * kS + col), u = {0, 0, 0, 0};
    if (m >= M) continue;
    z += bias;
    if constexpr (kGate) {
      u = *reinterpret_cast<const f32x4*>(strip + r * kS + col + 32);
      u += bias_up;
    }
    if (e.preact) {
      uint16_t* p = e.preact + m * (kGate ? 2 * (int64_t)N : N) + n;
      store_bf16x4(p, z, wide, left);
      if constexpr (kGate) store_bf16x4(p + N, u, wide, left);
    }
    f32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = activate<kAct>(z[k]);
      if constexpr (kGate) v[k] *= u[k];
    }
    if (e.residual) v += load_bf16x4(e.residual + m * e.residual_stride + n, wide, left);
    if (e.f32_out) store_f32x4(static_cast<float*>(y) + m * N + n, v, wide, left);
    else store_bf16x4(static_cast<uint16_t*>(y) + m * N + n, v, wide, left);
  }
}

// The whole tile of a wave: `strip` is its kStripBytes<TJ> of LDS, which no wave reads or
// writes otherwise any more; s multiplies the sums.
template <int TI, int TJ, bool kGate>
__device__ __forceinline__ void store_fused(const EpilogueArgs& e, void* y, float* strip, int M,
                                            int N, int m0, int n0, int lane, float s,
                                            const f32x16 (&acc)[TI][TJ]) {
  constexpr int kS = kStripStride<TJ>;
  constexpr int kAcross = (kGate ? 16 * TJ : 32 * TJ) / 4;
  const int lr = lane & 31, h = lane >> 5;
  const int n = n0 + 4 * (lane % kAcross);
  f32x4 bias = {0, 0, 0, 0}, bias_up = {0, 0, 0, 0};
  if (e.bias && n < N) {
    bias = load_bf16x4(e.bias + n, false, N - n);
    if (kGate) bias_up = load_bf16x4(e.bias + N + n, false, N - n);
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    if (m0 + 32 * i >= M) break;
#pragma unroll
    for (int t = 0; t < TJ; ++t)
#pragma unroll
      for (int a = 0; a < 16; ++a)
        strip[((a & 3) + 8 * (a >> 2) + 4 * h) * kS + 32 * t + lr] = acc[i][t][a] * s;
    const int m = m0 + 32 * i;
    switch (e.act) {
      case kActRelu: fused_strip<TJ, kGate, kActRelu>(e, y, strip, M, N, m, n0, lane, bias, bias_up); break;
      case kActGelu: fused_strip<TJ, kGate, kActGelu>(e, y, strip, M, N, m, n0, lane, bias, bias_up); break;
      case kActGeluTanh: fused_strip<TJ, kGate, kActGeluTanh>(e, y, strip, M, N, m, n0, lane, bias, bias_up); break;
      case kActSilu: fused_strip<TJ, kGate, kActSilu>(e, y, strip, M, N, m, n0, lane, bias, bias_up); break;
      default: fused_strip<TJ, kGate, kActNone>(e, y, strip, M, N, m, n0, lane, bias, bias_up);
    }
  }
}

}  // namespace gemm
}  // namespace fos
