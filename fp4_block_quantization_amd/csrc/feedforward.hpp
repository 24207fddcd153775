// Internal launch interface of the feed-forward operators: RMS norm with the residual's
// addition and a record as its output, products with an epilogue, and their backward passes.
#pragma once

#include "activation.hpp"

namespace fos {

constexpr int kMaxNormCols = 32768;      // a workgroup holds a row in registers

enum : int { kRecordNone, kRecordNVFP4, kRecordMXFP4 };

struct NormArgs {
  const uint16_t *x, *r;     // bf16 [M][K], row strides below (elements); r may be null
  int64_t x_stride, r_stride;
  const uint16_t* w;         // bf16 [K]
  int64_t M;
  int K;
  double eps;
  uint16_t* h;               // bf16 [M][K] or null
  float* rstd;               // [M] or null
  uint16_t* y;               // bf16 [M][K] or null
  int record;
  bool four_over_six;
  uint8_t *data, *scales;    // the record's
  float* t;                  // NVFP4: tensor scale, read (given) or written
  bool t_given;
  float* partials;           // kMaxPartials floats, where t is not given
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  const uint16_t *dy, *h, *w, *dh;   // bf16 [M][K], [M][K], [K], [M][K] or null
  const float* rstd;                 // [M]
  int64_t M;
  int K;
  uint16_t* dx;                      // bf16 [M][K]
  float* dw;                         // [K] or null
  float* partials;                   // [norm_bwd_partials][K]
};
int norm_bwd_partials(int64_t M, int K);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t s);

struct EpilogueBwdArgs {
  const uint16_t *dy, *z;    // bf16 [M][N], [M][N] (with a gate [M][2N])
  int64_t M, N;
  int act;
  bool gated;
  uint16_t* dz;              // like z
  float* dbias;              // [columns of z] or null
  float* t;                  // [1] or null: max |dz| / 2688
  float* partials;           // [epilogue_bwd_groups][columns of z] sums, then as many maxima
};
int64_t epilogue_bwd_grid(int64_t M, int64_t N);
int epilogue_bwd_groups(int64_t M, int64_t N);   // groups of rows with sums of their own
hipError_t launch_epilogue_bwd(const EpilogueBwdArgs& a, hipStream_t s);

// Y from Xq [M][K] and Wq [N][K], with a gate [2N][K]; wt and xt are null for MXFP4.
struct QLinearArgs {
  const uint8_t *xd, *xs, *wd, *ws;
  const float *xt, *wt;
  int64_t M, N, K;
  void* y;
  bool gated;
  EpilogueArgs e;
};
int64_t qlinear_epilogue_grid(const QLinearArgs& a);
hipError_t launch_qlinear_epilogue(const QLinearArgs& a, hipStream_t s);
int64_t mx_epilogue_grid(const QLinearArgs& a);
hipError_t launch_mx_epilogue(const QLinearArgs& a, hipStream_t s);

}  // namespace fos
