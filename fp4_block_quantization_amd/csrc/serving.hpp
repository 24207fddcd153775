// Internal launch interface of the token-serving operators (weight-only linear, paged
// key-value cache, paged attention of one new token) and the device helpers they share.
#pragma once

#include "activation.hpp"

namespace fos {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kCUs = 256;

// The workspace of the attention starts with counters of finished workgroups, 0 between
// launches; what is behind them is scratch.  One counter for each segment (a sequence and
// up to 16 query heads of a kv head), then one for each workgroup that runs at once.
constexpr int kCounters = 65536;
constexpr int kMaxPerCU = 3;
constexpr int kMaxResident = kMaxPerCU * kCUs;
constexpr size_t kCounterBytes = sizeof(uint32_t) * (kCounters + kMaxResident);

// Partial results pass from one workgroup to another on any XCD, each with an L2 of its
// own.  A release and an acquire fence at that scope write back and invalidate a whole L2
// (paged attention of 32 sequences of up to 8192 tokens: 262 us instead of 89); instead the
// few values that are passed are themselves accessed at device scope: the stores (relaxed
// atomics of 8 bytes) write through to memory and the loads read from there.  What orders them is
// that every thread waits until its stores are done (wait_stores), then the barrier, and
// only then one thread counts the workgroup: who reads the full count reads after all
// the stores.
__device__ __forceinline__ void store_shared(float* p, f32x2 v) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The loads, with the cache policy of device scope: 8 or 16 bytes at a byte offset of the
// `bytes` bytes at p (behind them: zeros).
constexpr int kDeviceScope = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t shared_floats(const float* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), 0, bytes, 0x27000);
}
__device__ __forceinline__ f32x2 load_shared2(__amdgpu_buffer_rsrc_t r, int offset) {
  return __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, offset, 0, kDeviceScope));
}
__device__ __forceinline__ f32x4 load_shared4(__amdgpu_buffer_rsrc_t r, int offset) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, kDeviceScope));
}
__device__ __forceinline__ void wait_stores() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Counts this workgroup as done with the work behind `counter`, once every thread's
// store_shared so far is done; true, for all threads, in the last of `count` workgroups
// (which has to put the counter back to 0 with reset_counter).  `before` is in LDS.
__device__ __forceinline__ bool last_to_finish(uint32_t* counter, int count, uint32_t& before) {
  wait_stores();                               // each thread's own, before the barrier
  __syncthreads();
  if (threadIdx.x == 0)
    before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return (int)before == count - 1;
}
__device__ __forceinline__ void reset_counter(uint32_t* counter) {
  if (threadIdx.x == 0)
    __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Weight-only linear: y[m][n] = t * sum_k x[m][k] deq(w)[n][k] (+ bias[n]), or an epilogue of it.
struct WLinearArgs {
  const uint16_t* x;       // bf16, row m at x + m * x_stride
  int64_t x_stride;        // elements
  const uint8_t* wd;       // [N][K/2]
  const uint8_t* ws;       // [N][K/16] E4M3 or [N][K/32] E8M0
  const float* wt;         // device fp32 (NVFP4) or null (MXFP4)
  const uint16_t* bias;    // bf16 [N] or null
  void* y;                 // [M][N] bf16 or fp32
  int64_t M, N, K;         // N: weight rows, with a gate two for each column of y
  bool mx, f32_out;
  // an epilogue other than the bias: none unless the caller says so
  bool fused = false, gated = false;
  EpilogueArgs e = {};     // its activation, residual and pre-activation
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
// Whether the head layout has few enough segments.
bool decode_heads_ok(int64_t Hq, int64_t heads);
size_t decode_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t dim);
hipError_t launch_paged_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace fos
