// RMS norm with the residual's addition, its output in bf16 or as a 4-bit record, and its
// backward pass.
//
//   h = RN_bf16(x + r),  rstd = RN(1 / sqrt(mean(h^2) + eps)),  y = RN_bf16(RN(h rstd) w)
// and the record is that of y, bit for bit fos_quantize's or fos_mx_quantize's.  The mean is
// taken in fp64 (a square of a bf16 value is exact in fp32, so only the sum rounds): rstd
// then does not depend on how a row is spread over lanes, and y, next to the rounding
// borders of a record, is the same whichever variant runs.
//
// Backward, with n = h rstd and g = dy w:
//   dx = RN_bf16(rstd (g - n mean(g n)) + dh),   dw = sum over rows of dy n  (fp32).
//
// Both are bound by memory, but for the second launch of an NVFP4 record under its own tensor
// scale, whose rounding of every block twice takes 77% of the VALU cycles.  8192 x 4096 with
// a residual: 36 us for h and the maxima (5.5 TB/s) and 26 for the record, 42 in one launch
// with a given tensor scale; backward 48 (5.6 TB/s) and 5 for dw's partial sums.  2047 x 12288
// with a residual to MXFP4 32 us (5.2 TB/s); one row of 4096 2.5.
//
// kLanes lanes share a row and keep it in registers, kBlocks blocks of 16 values each; lane l
// takes blocks l, l + kLanes, ..
#include "feedforward.hpp"

namespace fos {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Block {             // 16 bf16 values
  uint4 a, b;
};

__device__ __forceinline__ Block load_block(const uint16_t* p) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  return Block{q[0], q[1]};
}
__device__ __forceinline__ void store_block(uint16_t* p, const Block& v) {
  uint4* q = reinterpret_cast<uint4*>(p);
  q[0] = v.a;
  q[1] = v.b;
}
__device__ __forceinline__ Block pack_block(const float (&v)[16]) {
  return Block{make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])),
               make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]),
                          pack_bf16x2(v[12], v[13]), pack_bf16x2(v[14], v[15]))};
}
constexpr Block kZeroBlock = {};
// The same block, which the compiler takes for another: values unpacked from it are not kept
// in registers from (or for) elsewhere.
__device__ __forceinline__ Block again(Block v) {
  asm volatile("" : "+v"(v.a.x), "+v"(v.a.y), "+v"(v.a.z), "+v"(v.a.w));
  asm volatile("" : "+v"(v.b.x), "+v"(v.b.y), "+v"(v.b.z), "+v"(v.b.w));
  return v;
}
__device__ __forceinline__ void unpack_again(const Block& b, float (&v)[16]) {
  const Block c = again(b);
  unpack16(c.a, c.b, v);
}

// Sum over the kLanes lanes of a row, in all of them.  `part`: LDS for two rows in turn (one
// barrier a row), used where a row has more than one wave.
template <int kLanes, typename T>
__device__ __forceinline__ T row_sum(T v, T (*part)[16], int turn) {
  constexpr int kIn = kLanes < 64 ? kLanes : 64;
#pragma unroll
  for (int o = kIn / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (kLanes > 64) {
    T* p = part[turn & 1];
    if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
    __syncthreads();
    p += threadIdx.x / kLanes * (kLanes / 64);
    v = p[0];
#pragma unroll
    for (int w = 1; w < kLanes / 64; ++w) v += p[w];
  }
  return v;
}

// What a launch computes: the whole norm with its output in bf16 alone (kOutBF16), as an
// NVFP4 record under a given tensor scale, or as an MXFP4 record; or in two launches, where
// the tensor scale is that of the output: kOutMax (h, rstd and the maxima of |y|), then
// kOutSecond (the record, from h and rstd); or kOutOne, both, where one workgroup has all
// rows at once (1 x 4096: 4.0 us, 6.2 in two launches).
enum { kOutBF16, kOutNVFP4, kOutMXFP4, kOutMax, kOutSecond, kOutOne };

template <int kLanes, int kBlocks, int kOut, bool kRes>
__global__ __launch_bounds__(kLanes > 256 ? kLanes : 256)
void rmsnorm_kernel(NormArgs a, int npartials) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256, kRows = kThreads / kLanes;
  constexpr bool kNV = kOut == kOutNVFP4 || kOut == kOutSecond || kOut == kOutOne;
  __shared__ double part[2][16];
  __shared__ float2 tab[kNV ? kScaleTableSize : 1];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int blocks = a.K / 16;

  // the first row is on its way while the scale table is made, in the second launch every
  // row while the one before is quantized
  Block h[kBlocks], next[kBlocks];
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  const int64_t step = (int64_t)gridDim.x * kRows;
  auto load_row = [&](Block (&v)[kBlocks], int64_t at) {
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int b = lane + j * kLanes;
      v[j] = kZeroBlock;
      if (b < blocks) v[j] = load_block(a.x + at * a.x_stride + 16 * b);
    }
  };
  float next_rstd = 0.0f;
  if (row < a.M) {
    load_row(next, row);
    if (kOut == kOutSecond) next_rstd = a.rstd[row];
  }

  float u6 = 0.0f, u4 = 0.0f;
  if constexpr (kNV && kOut != kOutOne) {
    float t;
    if constexpr (kOut == kOutSecond) {
      // every workgroup reduces the maxima; a thread's maximum is over those 256 apart
      uint32_t m = 0;
      for (int i = threadIdx.x; i < npartials; i += kThreads)
        m = max(m, __float_as_uint(a.partials[i]));
      t = __uint_as_float(block_max_u32(m)) / kScaleDenom;
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.t = t;
    } else {
      t = *a.t;
    }
    build_scale_table(tab, t);
    u6 = tab[128].x;
    u4 = tab[128].y;
  }

  Block w[kBlocks];
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int b = lane + j * kLanes;
    w[j] = kZeroBlock;
    if (b < blocks) w[j] = load_block(a.w + 16 * b);
  }

  auto store_record = [&](const Block& y, int64_t at, int b) {
    float u[16];
    unpack16(y.a, y.b, u);
    const uint32_t none[16] = {};
    const Cand c = a.four_over_six ? quantize_block<true, false>(u, tab, u6, u4, none)
                                   : quantize_block<false, false>(u, tab, u6, u4, none);
    if (b < blocks) store_block_stream(a.data, a.scales, (at * blocks + b) * 8, at * blocks + b, c);
  };
  uint32_t top = 0;
  int turn = 0;
  for (bool first = true; row < a.M; row += step, ++turn, first = false) {
    float rstd = next_rstd;
    if (kOut != kOutSecond && !first) load_row(next, row);
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) h[j] = next[j];
    if (kOut == kOutSecond && row + step < a.M) {
      load_row(next, row + step);
      next_rstd = a.rstd[row + step];
    }
    if constexpr (kRes) {
      Block r[kBlocks];
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        const int b = lane + j * kLanes;
        r[j] = kZeroBlock;
        if (b < blocks) r[j] = load_block(a.r + row * a.r_stride + 16 * b);
      }
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        float u[16], v[16];
        unpack16(h[j].a, h[j].b, u);
        unpack16(r[j].a, r[j].b, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] += v[i];
        h[j] = pack_block(u);
      }
    }
    if constexpr (kOut != kOutSecond) {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        float u[16];
        unpack16(h[j].a, h[j].b, u);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const double d = u[i];
          ss = __builtin_fma(d, d, ss);
        }
      }
      ss = row_sum<kLanes>(ss, part, turn);
      rstd = (float)(1.0 / sqrt(ss / a.K + a.eps));
      if (a.rstd && lane == 0) a.rstd[row] = rstd;
      if (a.h) {
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
          const int b = lane + j * kLanes;
          if (b < blocks) store_block(a.h + row * a.K + 16 * b, h[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int b = lane + j * kLanes;
      float u[16], g[16];
      unpack_again(h[j], u);
      unpack_again(w[j], g);
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = u[i] * rstd * g[i];
      const Block y = pack_block(u);
      if (kOut != kOutSecond && a.y && b < blocks) store_block(a.y + row * a.K + 16 * b, y);
      if constexpr (kOut == kOutMax || kOut == kOutOne) top = pk_max_abs4(pk_max_abs4(top, y.a), y.b);
      if constexpr (kOut == kOutOne) h[j] = y;
      else if constexpr (kNV) store_record(y, row, b);
      if constexpr (kOut == kOutMXFP4) {
        // a block of 32 is this lane's and its neighbour's
        unpack16(y.a, y.b, u);
        float m = amax16(u);
        m = fmaxf(m, __shfl_xor(m, 1));
        const int ef = (int)(__float_as_uint(m) >> 23);
        const int e = ef == 0 ? -127 : max(ef - 129, -127);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t lo = 0, hi = 0;
        lo = cvt_pk_fp4<0>(lo, u[0] * inv, u[1] * inv);
        lo = cvt_pk_fp4<1>(lo, u[2] * inv, u[3] * inv);
        lo = cvt_pk_fp4<2>(lo, u[4] * inv, u[5] * inv);
        lo = cvt_pk_fp4<3>(lo, u[6] * inv, u[7] * inv);
        hi = cvt_pk_fp4<0>(hi, u[8] * inv, u[9] * inv);
        hi = cvt_pk_fp4<1>(hi, u[10] * inv, u[11] * inv);
        hi = cvt_pk_fp4<2>(hi, u[12] * inv, u[13] * inv);
        hi = cvt_pk_fp4<3>(hi, u[14] * inv, u[15] * inv);
        if (b < blocks) {
          __builtin_nontemporal_store(u32x2{lo, hi},
                                      reinterpret_cast<u32x2*>(a.data + (row * blocks + b) * 8));
          if ((lane & 1) == 0)
            __builtin_nontemporal_store((uint8_t)(e + 127), a.scales + (row * blocks + b) / 2);
        }
      }
    }
  }
  if constexpr (kOut == kOutMax) {
    top = block_max_u32(pk_max_to_f32_bits(top));
    if (threadIdx.x == 0) a.partials[blockIdx.x] = __uint_as_float(top);
  }
  if constexpr (kOut == kOutOne) {
    const float t = __uint_as_float(block_max_u32(pk_max_to_f32_bits(top))) / kScaleDenom;
    if (threadIdx.x == 0) *a.t = t;
    build_scale_table(tab, t);
    u6 = tab[128].x;
    u4 = tab[128].y;
    if (sub < a.M) {
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) store_record(h[j], sub, lane + j * kLanes);
    }
  }
}

template <int kLanes, int kBlocks, int kOut>
void launch_norm_kernel(const NormArgs& a, int grid, int npartials, hipStream_t s) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256;
  if (a.r) rmsnorm_kernel<kLanes, kBlocks, kOut, true><<<grid, kThreads, 0, s>>>(a, npartials);
  else rmsnorm_kernel<kLanes, kBlocks, kOut, false><<<grid, kThreads, 0, s>>>(a, npartials);
}

template <int kLanes, int kBlocks>
hipError_t launch_norm(NormArgs a, hipStream_t s) {
  constexpr int kRows = (kLanes > 256 ? kLanes : 256) / kLanes;
  const int64_t groups = (a.M + kRows - 1) / kRows;
  const int grid = (int)(groups < 2048 ? groups : 2048);
  if (a.record == kRecordNone) launch_norm_kernel<kLanes, kBlocks, kOutBF16>(a, grid, 0, s);
  else if (a.record == kRecordMXFP4) launch_norm_kernel<kLanes, kBlocks, kOutMXFP4>(a, grid, 0, s);
  else if (a.t_given) launch_norm_kernel<kLanes, kBlocks, kOutNVFP4>(a, grid, 0, s);
  else if (groups == 1) launch_norm_kernel<kLanes, kBlocks, kOutOne>(a, 1, 0, s);
  else {
    const int first = grid < kMaxPartials ? grid : kMaxPartials;
    launch_norm_kernel<kLanes, kBlocks, kOutMax>(a, first, 0, s);
    if (a.h) {
      a.x = a.h;
      a.x_stride = a.K;
      a.r = nullptr;
    }
    launch_norm_kernel<kLanes, kBlocks, kOutSecond>(a, first, first, s);
  }
  return hipGetLastError();
}

// No rows: the tensor scale of an empty tensor.
__global__ void zero_kernel(float* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// ------------------------------------------------------------------ backward
// A workgroup walks its rows and sums dw; partials[workgroup] is its sum.  With up to two blocks
// a lane the next row is on its way while one is computed, and dw is in registers.  With four (K
// above 16384) that does not fit, and what the compiler moved to scratch memory cost more than
// the copies: one row at a time and dw in LDS, each lane's own values (2048 x 32768: 132 us
// with dh, 4.1 TB/s; 258 with scratch).
template <int kLanes, int kBlocks, bool kRes>
__global__ __launch_bounds__(kLanes > 256 ? kLanes : 256, 2)
void rmsnorm_bwd_kernel(NormBwdArgs a) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256, kRows = kThreads / kLanes;
  __shared__ float part[2][16];
  __shared__ float sums[kRows > 1 ? kThreads * 16 : 1];
  constexpr bool kAhead = kBlocks <= 2;
  __shared__ float4 held[kAhead ? 1 : 4 * kBlocks][kAhead ? 1 : kThreads];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int blocks = a.K / 16;

  struct Row {
    Block h[kBlocks], dy[kBlocks], dh[kRes ? kBlocks : 1];
    float rstd;
  };
  auto load_row = [&](Row& r, int64_t row) {
    r.rstd = row < a.M ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int b = lane + j * kLanes;
      r.h[j] = r.dy[j] = kZeroBlock;
      if constexpr (kRes) r.dh[j] = kZeroBlock;
      if (b < blocks && row < a.M) {
        r.h[j] = load_block(a.h + row * a.K + 16 * b);
        r.dy[j] = load_block(a.dy + row * a.K + 16 * b);
        if constexpr (kRes) r.dh[j] = load_block(a.dh + row * a.K + 16 * b);
      }
    }
  };
  Row next;
  // the same number of rounds for all rows of a workgroup (they share barriers)
  int64_t first = (int64_t)blockIdx.x * kRows;
  const int64_t step = (int64_t)gridDim.x * kRows;
  if constexpr (kAhead) load_row(next, first + sub);

  Block w[kBlocks];
  float dw[kAhead ? kBlocks : 1][16];
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int b = lane + j * kLanes;
    w[j] = kZeroBlock;
    if (b < blocks) w[j] = load_block(a.w + 16 * b);
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < 16; ++i) dw[j][i] = 0.0f;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) held[4 * j + q][threadIdx.x] = make_float4(0, 0, 0, 0);
    }
  }
  const float inv_k = 1.0f / (float)a.K;
  int turn = 0;
  for (; first < a.M; first += step, ++turn) {
    const int64_t row = first + sub;
    Row r;
    if constexpr (kAhead) {
      r = next;
      if (first + step < a.M) load_row(next, row + step);
    } else {
      load_row(r, row);
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      float n[16], d[16], g[16];
      unpack_again(r.h[j], n);
      unpack_again(r.dy[j], d);
      unpack_again(w[j], g);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float dn = d[i] * (n[i] * r.rstd);
        if constexpr (kAhead) dw[j][i] += dn;
        else d[i] = dn;
        dot = __builtin_fmaf(dn, g[i], dot);
      }
      if constexpr (!kAhead) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4& v = held[4 * j + q][threadIdx.x];
          v = make_float4(v.x + d[4 * q], v.y + d[4 * q + 1], v.z + d[4 * q + 2], v.w + d[4 * q + 3]);
        }
      }
    }
    const float c = row_sum<kLanes>(dot, part, turn) * inv_k;
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      const int b = lane + j * kLanes;
      float n[16], d[16], g[16];
      unpack_again(r.h[j], n);
      unpack_again(r.dy[j], d);
      unpack_again(w[j], g);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        n[i] = r.rstd * __builtin_fmaf(-c, n[i] * r.rstd, d[i] * g[i]);
      if constexpr (kRes) {
        unpack_again(r.dh[j], d);
#pragma unroll
        for (int i = 0; i < 16; ++i) n[i] += d[i];
      }
      if (b < blocks && row < a.M) store_block(a.dx + row * a.K + 16 * b, pack_block(n));
    }
  }
  if (!a.dw) return;
  // one workgroup alone has dw itself
  float* out = gridDim.x == 1 ? a.dw : a.partials + (int64_t)blockIdx.x * a.K;
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int b = lane + j * kLanes;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[i * kThreads + threadIdx.x] = dw[j][i];
      __syncthreads();
      // thread (lane, sub) joins the rows' sums of 16 / kRows of its lane's values
      constexpr int kEach = 16 / kRows;
      float v[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        v[e] = 0.0f;
#pragma unroll
        for (int q = 0; q < kRows; ++q) v[e] += sums[(sub * kEach + e) * kThreads + q * kLanes + lane];
      }
      if (b < blocks) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) out[16 * b + sub * kEach + e] = v[e];
      }
    } else if (b < blocks) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        float4 v;
        if constexpr (kAhead) v = make_float4(dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]);
        else v = held[4 * j + i / 4][threadIdx.x];
        *reinterpret_cast<float4*>(out + 16 * b + i) = v;
      }
    }
  }
}

// dw[k] = sum over n partial rows, in their order within 32 groups, then over the groups:
// 8 lanes to a row's 32 columns.
__global__ __launch_bounds__(256) void column_sum_kernel(const float* __restrict__ p, int n, int K,
                                                         float* __restrict__ dw) {
  __shared__ float4 part[32][8];
  const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int k = (int)blockIdx.x * 32 + 4 * c;
  float4 v = make_float4(0, 0, 0, 0);
  if (k < K) {
#pragma unroll 8
    for (int i = g; i < n; i += 32) {
      const float4 q = *reinterpret_cast<const float4*>(p + (int64_t)i * K + k);
      v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
    }
  }
  part[g][c] = v;
  __syncthreads();
  if (g == 0 && k < K) {
    for (int i = 1; i < 32; ++i) {
      const float4 q = part[i][c];
      v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
    }
    *reinterpret_cast<float4*>(dw + k) = v;
  }
}

template <int kLanes, int kBlocks>
hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t s) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256;
  const int grid = norm_bwd_partials(a.M, a.K);
  if (a.dh) rmsnorm_bwd_kernel<kLanes, kBlocks, true><<<grid, kThreads, 0, s>>>(a);
  else rmsnorm_bwd_kernel<kLanes, kBlocks, false><<<grid, kThreads, 0, s>>>(a);
  if (a.dw && grid > 1) column_sum_kernel<<<(a.K + 31) / 32, 256, 0, s>>>(a.partials, grid, a.K, a.dw);
  return hipGetLastError();
}

// Lanes of a row: a wave where its four blocks a lane hold the row, else more waves; few rows
// get more lanes.
int lanes_of(int64_t M, int K) {
  if (K <= 512) return 16;
  if (K > 16384) return 512;
  return K > 4096 || M < 1024 ? 256 : 64;
}
// Two blocks a lane where it can be.
int bwd_lanes_of(int64_t M, int K) {
  if (K <= 512) return 16;
  if (M < 1024 && K <= 8192) return 256;
  return K <= 2048 ? 64 : K <= 4096 ? 128 : K <= 8192 ? 256 : 512;
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.M == 0) {
    if (a.record != kRecordNVFP4 || a.t_given) return hipSuccess;
    zero_kernel<<<1, 64, 0, s>>>(a.t, 1);
    return hipGetLastError();
  }
  // four rows fit one workgroup, which then needs no second launch (4 x 1024: 4.4 us, in two
  // launches with 256 lanes a row 6.8; 4 x 4096: 6.9 and 6.7, called from Python 14.5 and 17.5)
  const bool one = a.record == kRecordNVFP4 && !a.t_given && a.M <= 4 && a.K > 512 && a.K <= 4096;
  const int lanes = one && a.M > 1 ? 64 : lanes_of(a.M, a.K), per = (a.K / 16 + lanes - 1) / lanes;
  switch (lanes) {
    case 16: return per <= 1 ? launch_norm<16, 1>(a, s) : launch_norm<16, 2>(a, s);
    case 64: return per <= 2 ? launch_norm<64, 2>(a, s) : launch_norm<64, 4>(a, s);
    case 256:
      return per <= 1 ? launch_norm<256, 1>(a, s) : per <= 2 ? launch_norm<256, 2>(a, s)
           : per <= 3 ? launch_norm<256, 3>(a, s) : launch_norm<256, 4>(a, s);
    default: return launch_norm<512, 4>(a, s);
  }
}

// Workgroups of the backward pass, each with a partial dw: what runs at once (two waves to a
// SIMD), but at least four rounds of rows to each, down to one workgroup to a CU.  Up to two
// rounds are one workgroup, whose sums are dw itself: no second launch (2 x 4096: 4.7 us, 6.0 with
// two launches; four rounds of 64 x 512 9.5 and 6.8).
int norm_bwd_partials(int64_t M, int K) {
  const int lanes = bwd_lanes_of(M, K), rows = lanes > 256 ? 1 : 256 / lanes;
  const int64_t groups = (M + rows - 1) / rows, most = lanes > 256 ? 256 : 512;
  if (groups <= 2) return 1;
  const int64_t want = groups / 4 < 256 ? 256 : groups / 4 < most ? groups / 4 : most;
  return (int)(groups < want ? groups : want);
}

hipError_t launch_rmsnorm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.M == 0) {
    if (!a.dw) return hipSuccess;
    zero_kernel<<<(a.K + 255) / 256, 256, 0, s>>>(a.dw, a.K);
    return hipGetLastError();
  }
  const int lanes = bwd_lanes_of(a.M, a.K), per = (a.K / 16 + lanes - 1) / lanes;
  switch (lanes) {
    case 16: return per <= 1 ? launch_bwd<16, 1>(a, s) : launch_bwd<16, 2>(a, s);
    case 64: return launch_bwd<64, 2>(a, s);
    case 128: return launch_bwd<128, 2>(a, s);
    case 256: return per <= 1 ? launch_bwd<256, 1>(a, s) : launch_bwd<256, 2>(a, s);
    default: return per <= 2 ? launch_bwd<512, 2>(a, s) : launch_bwd<512, 4>(a, s);
  }
}

}  // namespace fos
