// Paged key-value cache: append rows of new tokens to their slots and read slots back.
//
// The cache is [page][kv head][token of the page][value], so a page holds each head's
// tokens in one run; an NVFP4 page of a head is an NVFP4 record [page_size][dim] (16
// values of a row per E4M3 block scale, static fp32 tensor scales for all of K and all
// of V).  Slot = page * page_size + token of the page; a slot outside the cache is
// skipped (append) or read as zeros (gather).
//
// Memory bounds it: 8192 tokens of 8 heads of 128, NVFP4, take 19.6 us for both, 4.4 TB/s of
// the 5.1 that a large copy reaches; few tokens (32: 4.8 us for both) take their two launches.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;

// Divisions of the index arithmetic as products with ceil(2^k / d): exact where the
// dividend times d stays below 2^k.
struct Div64 {                  // dividend < 2^40, d < 2^24
  uint64_t magic;
  explicit Div64(uint64_t d) : magic(~(uint64_t)0 / d + 1) {}
  __device__ __forceinline__ uint64_t operator()(uint64_t x) const { return __umul64hi(x, magic); }
};
struct Div32 {                  // dividend * d < 2^32
  uint32_t magic;
  explicit Div32(uint32_t d) : magic(~(uint32_t)0 / d + 1) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return __umulhi(x, magic); }
};

// One thread per kValues consecutive values of a row; blockIdx.y 0: K, 1: V.
struct Plan {
  KVRowsArgs a;
  int64_t n;                    // threads of K
  uint32_t per, units;          // threads of a token (at most 65536 * 32), of a row
  Div64 by_per, by_page;
  Div32 by_units;
  Plan(const KVRowsArgs& args, int values)
      : a(args), n(args.T * args.c.heads * (args.c.dim / values)),
        per((uint32_t)(args.c.heads * (args.c.dim / values))),
        units((uint32_t)(args.c.dim / values)), by_per(per), by_page((uint64_t)args.c.page_size),
        by_units(units) {}
  dim3 grid() const { return dim3((uint32_t)((n + kThreads - 1) / kThreads), 2); }
};

// What a thread works on: unit `unit` (of per) of token tok, and its place in the cache in
// units, or -1 for a slot outside it.
struct Where {
  int64_t tok, at;
  uint32_t unit;
};
__device__ __forceinline__ Where locate(const Plan& p, int64_t i) {
  Where w;
  w.tok = (int64_t)p.by_per((uint64_t)i);
  w.unit = (uint32_t)(i - w.tok * p.per);
  const KVCacheArgs& c = p.a.c;
  const int64_t slot = p.a.slots[w.tok];
  w.at = -1;
  if (slot >= 0 && slot < c.num_pages * c.page_size) {
    const int64_t page = (int64_t)p.by_page((uint64_t)slot);
    const uint32_t head = p.by_units(w.unit);
    const int64_t row = (page * c.heads + head) * c.page_size + (slot - page * c.page_size);
    w.at = row * p.units + (w.unit - head * p.units);
  }
  return w;
}

typedef u32x4 v4u;

// 16 values: one block.  The input is loaded before the workgroup's table of scales is
// built.  Cached loads: new rows come out of the projection before (8192 tokens of 8 heads
// of 128, append and gather: 19.5 us, with non-temporal loads 22.9).
template <bool k46>
__global__ __launch_bounds__(kThreads) void append_nvfp4_kernel(Plan p) {
  __shared__ float2 tab[kScaleTableSize];
  const KVRowsArgs& a = p.a;
  const bool is_v = blockIdx.y != 0;
  const float t = is_v ? a.c.vt[0] : a.c.kt[0];
  const int64_t i = min((int64_t)blockIdx.x * kThreads + threadIdx.x, p.n - 1);
  const Where w = locate(p, i);      // threads past the last do the last once more
  const v4u* src = reinterpret_cast<const v4u*>((is_v ? a.v + w.tok * a.v_stride
                                                      : a.k + w.tok * a.k_stride) + 16 * w.unit);
  const v4u l0 = src[0], l1 = src[1];
  build_scale_table(tab, t);
  if (w.at < 0) return;
  float v[16];
  unpack16(make_uint4(l0.x, l0.y, l0.z, l0.w), make_uint4(l1.x, l1.y, l1.z, l1.w), v);
  const uint32_t none[16] = {};
  const Cand c = quantize_block<k46, false>(v, tab, tab[128].x, tab[128].y, none);
  *reinterpret_cast<uint2*>((is_v ? a.c.v : a.c.k) + 8 * w.at) = make_uint2(c.lo, c.hi);
  (is_v ? a.c.vs : a.c.ks)[w.at] = (uint8_t)c.s;
}

// 8 values.
__global__ __launch_bounds__(kThreads) void append_bf16_kernel(Plan p) {
  const KVRowsArgs& a = p.a;
  const bool is_v = blockIdx.y != 0;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.n) return;
  const Where w = locate(p, i);
  if (w.at < 0) return;
  const uint16_t* src = (is_v ? a.v + w.tok * a.v_stride : a.k + w.tok * a.k_stride) + 8 * w.unit;
  reinterpret_cast<v4u*>(is_v ? a.c.v : a.c.k)[w.at] = *reinterpret_cast<const v4u*>(src);
}

// 8 values.
template <bool kNVFP4>
__global__ __launch_bounds__(kThreads) void gather_kernel(Plan p) {
  const KVRowsArgs& a = p.a;
  const bool is_v = blockIdx.y != 0;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.n) return;
  const Where w = locate(p, i);
  v4u o = {0, 0, 0, 0};
  if (w.at >= 0) {
    if (kNVFP4) {
      const uint32_t q = reinterpret_cast<const uint32_t*>(is_v ? a.c.v : a.c.k)[w.at];
      const float d = e4m3_decode((is_v ? a.c.vs : a.c.ks)[w.at >> 1]) * (is_v ? a.c.vt[0] : a.c.kt[0]);
      const f32x2 e0 = cvt_pk_f32_fp4<0>(q), e1 = cvt_pk_f32_fp4<1>(q);
      const f32x2 e2 = cvt_pk_f32_fp4<2>(q), e3 = cvt_pk_f32_fp4<3>(q);
      o = v4u{pack_bf16x2(e0.x * d, e0.y * d), pack_bf16x2(e1.x * d, e1.y * d),
              pack_bf16x2(e2.x * d, e2.y * d), pack_bf16x2(e3.x * d, e3.y * d)};
    } else {
      o = reinterpret_cast<const v4u*>(is_v ? a.c.v : a.c.k)[w.at];
    }
  }
  uint16_t* dst = (is_v ? a.v + w.tok * a.v_stride : a.k + w.tok * a.k_stride) + 8 * w.unit;
  *reinterpret_cast<v4u*>(dst) = o;
}

}  // namespace

hipError_t launch_kv_append(const KVRowsArgs& a, hipStream_t s) {
  const Plan p(a, a.c.nvfp4 ? 16 : 8);
  if (!a.c.nvfp4) append_bf16_kernel<<<p.grid(), kThreads, 0, s>>>(p);
  else if (a.four_over_six) append_nvfp4_kernel<true><<<p.grid(), kThreads, 0, s>>>(p);
  else append_nvfp4_kernel<false><<<p.grid(), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv_gather(const KVRowsArgs& a, hipStream_t s) {
  const Plan p(a, 8);
  if (a.c.nvfp4) gather_kernel<true><<<p.grid(), kThreads, 0, s>>>(p);
  else gather_kernel<false><<<p.grid(), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace fos
