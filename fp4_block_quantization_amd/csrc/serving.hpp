// Internal launch interface of the token-serving operators (weight-only linear, paged
// key-value cache, paged attention of one new token) and the device helpers they share.
#pragma once

#include "device_common.hpp"

namespace fos {

// Weight-only linear: y[m][n] = t * sum_k x[m][k] deq(w)[n][k] (+ bias[n]).
struct WLinearArgs {
  const uint16_t* x;       // bf16, row m at x + m * x_stride
  int64_t x_stride;        // elements
  const uint8_t* wd;       // [N][K/2]
  const uint8_t* ws;       // [N][K/16] E4M3 or [N][K/32] E8M0
  const float* wt;         // device fp32 (NVFP4) or null (MXFP4)
  const uint16_t* bias;    // bf16 [N] or null
  void* y;                 // [M][N] bf16 or fp32
  int64_t M, N, K;
  bool mx, f32_out;
};
int64_t wlinear_threads(const WLinearArgs& a);   // work-items of the launch
hipError_t launch_wlinear(const WLinearArgs& a, hipStream_t s);

// Paged key-value cache: [page][kv head][token of the page][value].
struct KVCacheArgs {
  bool nvfp4;
  int64_t num_pages;
  int page_size, heads, dim;
  uint8_t *k, *v;          // bf16 values or nibbles
  uint8_t *ks, *vs;        // E4M3 block scales (NVFP4)
  const float *kt, *vt;    // device fp32 tensor scales (NVFP4)
};
struct KVRowsArgs {
  KVCacheArgs c;
  const int64_t* slots;    // [T]
  int64_t T;
  uint16_t *k, *v;         // bf16 rows: [token][head][dim], token stride below (elements)
  int64_t k_stride, v_stride;
  bool four_over_six;      // append only
};
hipError_t launch_kv_append(const KVRowsArgs& a, hipStream_t s);
hipError_t launch_kv_gather(const KVRowsArgs& a, hipStream_t s);

struct DecodeArgs {
  KVCacheArgs c;
  const uint16_t* q;       // bf16 [B][Hq][dim], sequence stride q_stride (elements)
  int64_t q_stride;
  int B, Hq, G;            // G = Hq / heads: query heads per kv head
  const int32_t* table;    // [B][pages_per_seq], row stride table_stride
  int64_t table_stride;
  int pages_per_seq;
  const int32_t* lens;     // [B]
  float scale;
  int64_t window;          // 0: every token
  uint16_t* out;           // bf16 [B][Hq][dim]
  float* lse;              // [B][Hq] or null
  void* ws;
};
// Whether the head layout has few enough segments, and the bytes at the start of the
// workspace that are 0 between launches.
bool decode_heads_ok(int64_t Hq, int64_t heads);
size_t decode_counter_bytes();
size_t decode_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t dim);
hipError_t launch_paged_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace fos
