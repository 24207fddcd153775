// Backward pass of a product's epilogue: from dY and the pre-activation Z,
//   dZ = dY act'(Z),   with a gate  dZ_gate = dY Z_up act'(Z_gate),  dZ_up = dY act(Z_gate),
// dbias = column sums of dZ before its rounding (fp32), and max |dZ| / 2688, the tensor scale
// with which dZ is quantized next.
//
// Bound by memory: 4096 x 12288 with gelu_tanh 59 us (5.1 TB/s; VALU busy 66%), the sums of
// dbias joined in 5 more (4096 x 12287, value by value: 92).  A wave takes 64 x kCols columns (one 16-byte load a lane, or one value
// where rows are not aligned for that) of every fourth row of the workgroup's rows, and keeps
// the columns' sums in registers; the workgroup's four waves join theirs in LDS, and a
// second launch joins the groups of rows, always in the same order.
#include "feedforward.hpp"

namespace fos {

namespace {

// Rows of one group: few enough for about 2048 workgroups, 16 at least, so that the partial
// sums are little beside dZ (one fp32 for 16 bf16 values or more).  Up to 32 rows are one
// group, whose sums are dbias itself: no second launch, if there is no tensor scale to join
// (16 x 4096: 4.0 us, 5.9 with two launches; 32 x 12288: 5.8 and 6.1).
int rows_of_group(int64_t M, int64_t N) {
  if (M <= 32) return 32;
  const int64_t strips = (N + 511) / 512;
  int64_t rows = (M * strips + 2047) / 2048;
  rows = (rows + 15) / 16 * 16;
  return (int)(rows < 16 ? 16 : rows > (1 << 20) ? 1 << 20 : rows);
}

template <int kCols>
__device__ __forceinline__ void load_cols(const uint16_t* p, float (&v)[kCols]) {
  if constexpr (kCols == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
  } else {
    v[0] = bf16_lo(*p);
  }
}
// Stores the values rounded, and takes their maximum into `top` (packed pairs).
template <int kCols>
__device__ __forceinline__ void store_cols(uint16_t* p, const float (&v)[kCols], uint32_t& top) {
  if constexpr (kCols == 8) {
    const uint4 q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    *reinterpret_cast<uint4*>(p) = q;
    top = pk_max_abs4(top, q);
  } else {
    const uint32_t q = pack_bf16x2(v[0], 0.0f);
    *p = (uint16_t)q;
    top = pk_max_abs(top, q);
  }
}

template <int kAct, bool kGated, int kCols>
__global__ __launch_bounds__(256) void epilogue_bwd_kernel(EpilogueBwdArgs a, int group_rows,
                                                           int strips) {
  constexpr int kHalves = kGated ? 2 : 1;
  __shared__ float sums[4][kHalves][64 * kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = blockIdx.x / strips, strip = blockIdx.x % strips;
  const int64_t n = (int64_t)strip * (64 * kCols) + kCols * lane, width = kHalves * a.N;
  const int64_t first = (int64_t)group * group_rows, last = min(first + group_rows, a.M);
  const bool in = n < a.N;
  float sum[kHalves][kCols] = {};
  uint32_t top = 0;
  if (in) {
#pragma unroll 2
    for (int64_t m = first + wave; m < last; m += 4) {
      float dy[kCols], z[kCols], d[kCols];
      load_cols(a.dy + m * a.N + n, dy);
      load_cols(a.z + m * width + n, z);
      if constexpr (kGated) {
        float up[kCols], du[kCols];
        load_cols(a.z + m * width + a.N + n, up);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          float f, df;
          activate_slope<kAct>(z[i], f, df);
          d[i] = dy[i] * up[i] * df;
          du[i] = dy[i] * f;
          sum[0][i] += d[i];
          sum[kHalves - 1][i] += du[i];
        }
        store_cols(a.dz + m * width + a.N + n, du, top);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          float f, df;
          activate_slope<kAct>(z[i], f, df);
          d[i] = dy[i] * df;
          sum[0][i] += d[i];
        }
      }
      store_cols(a.dz + m * width + n, d, top);
    }
  }
  if (a.t) {
    top = block_max_u32(pk_max_to_f32_bits(top));
    // the maxima are behind the sums
    if (threadIdx.x == 0)
      a.partials[(a.dbias ? (int64_t)(gridDim.x / strips) * width : 0) + blockIdx.x] =
          __uint_as_float(top);
  }
  if (!a.dbias) return;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int i = 0; i < kCols; ++i) sums[wave][h][i * 64 + lane] = sum[h][i];
  __syncthreads();
  for (int i = wave; i < kHalves * kCols; i += 4) {
    const int h = i / kCols, c = i % kCols;
    if (!in) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += sums[w][h][c * 64 + lane];
    (gridDim.x == strips ? a.dbias : a.partials)[(int64_t)group * width + h * a.N + n + c] = v;
  }
}

// The groups' sums joined, 64 columns to a workgroup, whose four waves take every fourth
// group; the last workgroup joins the maxima.
__global__ __launch_bounds__(256) void epilogue_join_kernel(const float* __restrict__ p, int groups,
                                                            int64_t width, int nmax,
                                                            float* __restrict__ dbias,
                                                            float* __restrict__ t) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (t && blockIdx.x == gridDim.x - 1) {
    const float* q = p + (dbias ? groups * width : 0);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < nmax; i += 256) m = max(m, __float_as_uint(q[i]));
    m = block_max_u32(m);
    if (threadIdx.x == 0) *t = __uint_as_float(m) / kScaleDenom;
    return;
  }
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (n < width) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 4) v += p[g * width + n];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && n < width) dbias[n] = part[0][lane] + part[1][lane] + part[2][lane] + part[3][lane];
}

bool wide(const EpilogueBwdArgs& a) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.z) |
                      reinterpret_cast<uintptr_t>(a.dz);
  return a.N % 8 == 0 && p % 16 == 0;
}

template <int kAct>
void launch_act(const EpilogueBwdArgs& a, int rows, int groups, int64_t grid8, int64_t grid1,
                int strips8, int strips1, hipStream_t s) {
  if (wide(a)) {
    if (a.gated) epilogue_bwd_kernel<kAct, true, 8><<<grid8, 256, 0, s>>>(a, rows, strips8);
    else epilogue_bwd_kernel<kAct, false, 8><<<grid8, 256, 0, s>>>(a, rows, strips8);
  } else {
    if (a.gated) epilogue_bwd_kernel<kAct, true, 1><<<grid1, 256, 0, s>>>(a, rows, strips1);
    else epilogue_bwd_kernel<kAct, false, 1><<<grid1, 256, 0, s>>>(a, rows, strips1);
  }
}

}  // namespace

int epilogue_bwd_groups(int64_t M, int64_t N) {
  const int rows = rows_of_group(M, N);
  return (int)((M + rows - 1) / rows);
}

// Workgroups where every lane takes one column (the most that a shape needs).
int64_t epilogue_bwd_grid(int64_t M, int64_t N) {
  return (int64_t)epilogue_bwd_groups(M, N) * ((N + 63) / 64);
}

hipError_t launch_epilogue_bwd(const EpilogueBwdArgs& a, hipStream_t s) {
  const int groups = epilogue_bwd_groups(a.M, a.N);
  const int strips8 = (int)((a.N + 511) / 512), strips1 = (int)((a.N + 63) / 64);
  const int64_t grid8 = (int64_t)groups * strips8, grid1 = epilogue_bwd_grid(a.M, a.N);
  if (a.M > 0) {
    const int rows = rows_of_group(a.M, a.N);
    switch (a.act) {
      case kActRelu: launch_act<kActRelu>(a, rows, groups, grid8, grid1, strips8, strips1, s); break;
      case kActGelu: launch_act<kActGelu>(a, rows, groups, grid8, grid1, strips8, strips1, s); break;
      case kActGeluTanh: launch_act<kActGeluTanh>(a, rows, groups, grid8, grid1, strips8, strips1, s); break;
      case kActSilu: launch_act<kActSilu>(a, rows, groups, grid8, grid1, strips8, strips1, s); break;
      default: launch_act<kActNone>(a, rows, groups, grid8, grid1, strips8, strips1, s);
    }
  }
  if (a.M == 0 && !a.dbias && !a.t) return hipSuccess;
  const int64_t width = a.gated ? 2 * a.N : a.N;
  const bool sums = a.dbias && groups != 1;   // of no rows: zeros
  const int64_t join = (sums ? (width + 63) / 64 : 0) + (a.t ? 1 : 0);
  if (join)
    epilogue_join_kernel<<<join, 256, 0, s>>>(a.partials, groups, width,
                                              (int)(wide(a) ? grid8 : grid1), a.dbias, a.t);
  return hipGetLastError();
}

}  // namespace fos
