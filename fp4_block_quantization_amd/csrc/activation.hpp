// Activation functions of the feed-forward operators, and the epilogue of a product: bias,
// activation, gate, residual, and the pre-activation kept for the backward pass.
//
//   none z;  relu max(z, 0);  silu z s(z), s(z) = 1 / (1 + e^-z);
//   gelu z F(z), F the standard normal distribution function;
//   gelu_tanh z s(2 sqrt(2/pi) (z + 0.044715 z^3)), which is z (1 + tanh(..)) / 2.
//
// All in fp32 on the hardware's exponential and reciprocal (1 ulp each).
#pragma once

#include "device_common.hpp"

namespace fos {

enum : int { kActNone, kActRelu, kActGelu, kActGeluTanh, kActSilu, kActs };

constexpr float kLog2e = 1.44269504f;
constexpr float kTanhC = 1.59576912f;      // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution's upper tail at |z|: erfc(x) / 2 at x = |z| / sqrt 2, as
// e^(-x^2) t P(t) with t = 1 / (1 + 0.44 x).  P is a least-maximum fit of degree 7 to
// e^(x^2) erfc(x) / (2 t) over x in [0, 10] (beyond, e^(-x^2) is 0 in fp32): relative error
// 1.9e-7, and t P 5e-7 with fp32's roundings.  The exponent carries three roundings (z^2, the
// constant, their product), 1.5 z^2 u of e with u = 2^-24: the tail is within (1.5 z^2 + 20) u
// (found: 8e-7 up to |z| = 4, 8e-6 at 12.9; half a step of bf16 is 4e-3).  To multiply what the
// roundings leave into e again would take six operations more for each value.
// e: e^(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float& e) {
  e = fast_exp2(z * z * (-0.5f * kLog2e));
  const float t = fast_rcp(__builtin_fmaf(fabsf(z), 0.44f * 0.70710678f, 1.0f));
  float p = 0.03561196103692055f;
  p = __builtin_fmaf(p, t, -0.13897496461868286f);
  p = __builtin_fmaf(p, t, 0.14834542572498322f);
  p = __builtin_fmaf(p, t, -0.010091908276081085f);
  p = __builtin_fmaf(p, t, 0.10790695995092392f);
  p = __builtin_fmaf(p, t, 0.10865651816129684f);
  p = __builtin_fmaf(p, t, 0.12443563342094421f);
  p = __builtin_fmaf(p, t, 0.12411047518253326f);
  return p * t * e;
}

// 1 / (1 + e^-u)
__device__ __forceinline__ float sigmoid(float u) {
  return fast_rcp(1.0f + fast_exp2(u * -kLog2e));
}

template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == kActRelu) return z < 0.0f ? 0.0f : z;   // a NaN stays, which fmaxf drops
  if constexpr (kAct == kActGelu) {
    float e;
    const float q = normal_tail(z, e);
    return z * (z < 0.0f ? q : 1.0f - q);
  }
  if constexpr (kAct == kActGeluTanh)
    return z * sigmoid(z * __builtin_fmaf(z * z, kTanhC * kTanhCubic, kTanhC));
  if constexpr (kAct == kActSilu) return z * sigmoid(z);
  return z;
}

// The same with the activation known at run time only (the same for all threads).
__device__ __forceinline__ float activate(int act, float z) {
  switch (act) {
    case kActRelu: return activate<kActRelu>(z);
    case kActGelu: return activate<kActGelu>(z);
    case kActGeluTanh: return activate<kActGeluTanh>(z);
    case kActSilu: return activate<kActSilu>(z);
    default: return z;
  }
}

// Value and slope.  s(u) and s(-u) come from e^-|u|, which does not overflow; z^2 is taken
// of a z within +-10^6 (there the slope is 0 or 1).  fminf and fmaxf make a number of a
// NaN, which value and slope then have from z itself.
template <int kAct>
__device__ __forceinline__ void activate_slope(float z, float& f, float& df) {
  if constexpr (kAct == kActNone) {
    f = z;
    df = 1.0f;
  } else if constexpr (kAct == kActRelu) {
    f = z < 0.0f ? 0.0f : z;
    df = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (kAct == kActGelu) {
    float e;
    const float q = normal_tail(z, e);
    const float p = z < 0.0f ? q : 1.0f - q;
    f = z * p;
    df = __builtin_fmaf(fminf(fmaxf(z, -1e6f), 1e6f), e * 0.39894228f, p);   // z / sqrt(2 pi) e^..
  } else {
    const float zc = fminf(fmaxf(z, -1e6f), 1e6f);
    const float z2 = zc * zc;
    const float u = kAct == kActSilu ? z : z * __builtin_fmaf(z2, kTanhC * kTanhCubic, kTanhC);
    const float du = kAct == kActSilu ? 1.0f : __builtin_fmaf(z2, 3.0f * kTanhC * kTanhCubic, kTanhC);
    const float e = fast_exp2(fabsf(u) * -kLog2e), r = fast_rcp(1.0f + e), er = e * r;
    const float p = u < 0.0f ? er : r;
    f = z * p;
    df = __builtin_fmaf(zc * du, er * r, p);
  }
}

// Y = act(Z) + residual, or with a gate Y = act(Z_gate) * Z_up + residual.
struct EpilogueArgs {
  const uint16_t* bias;      // bf16 [weight rows] or null
  const uint16_t* residual;  // bf16 [M][N], row stride below (elements), or null
  int64_t residual_stride;
  uint16_t* preact;          // bf16 [M][weight rows] or null
  int act;
  bool f32_out;
  bool pair, quad;           // two, four columns can be accessed at once (quad: of bias, too)
};
// Largest sizes that the GEMM kernels' epilogue addresses.
constexpr int64_t kMaxEpilogueCols = 1 << 20, kMaxResidualStride = 1 << 22;

}  // namespace fos
