// Weight-only quantized linear layer: bf16 activations times a 4-bit weight record,
//   y[m][n] = t * sum_k x[m][k] E(w[n][k]) D(s[n][k / block]) + bias[n].
// The weight is read once for each tile of activation rows (up to 64); with few rows its
// bytes bound the call (x and y are small beside it).
// Measured, a launch included (1.8 us when empty), where a plain read of the weight takes
// 5.5 us: 1 x 12288 x 4096 NVFP4 8.0 to 8.4 us, 16 x 12288 x 4096 9.1 us; 1 x 256 x 256 2.8
// us.  With more rows the conversions and the passage through LDS bound it: 61 x 4099 x 4112
// 12.2 us (of 256 CUs 172 have work), 64 x 12288 x 4096 17 us.
//
// Matrix form: E2M1 x E4M3 has at most 6 significant bits and E2M1 x 2^e two, so weights
// are exact in bf16, products are exact in fp32, and every sum is fp32; y is rounded once.
// Two kernels, by the number of activation rows (shape_of): few on 4x4x4 products, where a
// lane keeps a weight row to itself, and more on 16x16x32 tiles, where a weight is
// converted once for the 16, 32 or 64 activation rows of a tile.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kChunk = 128;   // values of the inner dimension per wave and step

// Weight rows are K / 2 bytes apart: 8-byte alignment (K % 16 == 0).
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight nibbles times a block scale as bf16: through fp32 for an E4M3 scale (a factor of
// up to four significant bits), in the conversion itself for a power of two.
template <bool kMX>
__device__ __forceinline__ u32x4 dequant8(uint32_t w, float d) {
  if constexpr (kMX) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, d, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, d, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, d, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, d, 3))};
  } else {
    const f32x2 a = cvt_pk_f32_fp4<0>(w), b = cvt_pk_f32_fp4<1>(w);
    const f32x2 c = cvt_pk_f32_fp4<2>(w), e = cvt_pk_f32_fp4<3>(w);
    return u32x4{pack_bf16x2(a.x * d, a.y * d), pack_bf16x2(b.x * d, b.y * d),
                 pack_bf16x2(c.x * d, c.y * d), pack_bf16x2(e.x * d, e.y * d)};
  }
}
// The scales of 32 values: two E4M3 bytes, or one E8M0 byte (2^-127 is subnormal in fp32).
template <bool kMX>
__device__ __forceinline__ f32x2 scale_values(uint32_t w) {
  if constexpr (kMX) {
    const float d = __uint_as_float(max(w << 23, 0x400000u));
    return f32x2{d, d};
  } else {
    return __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  }
}

// ---- more activation rows: 16x16x32 tiles -------------------------------------------
// A wave takes 16 NT weight rows (A operand) by 16 MT activation rows (B operand) and walks
// the inner dimension in chunks of 128; the waves of a workgroup share the tile and split
// the inner dimension.  Lane (r = lane % 16, q = lane / 16) supplies to step j of a chunk
// the values 32 q + 8 j .. + 7 of row r: 16 contiguous bytes of a weight row.  Loaded like
// that, neighbouring lanes would sit in different rows and cost the address unit a line
// each (18.8 us at 16 x 12288 x 4096), so weights and activations are loaded in memory
// order and go through the wave's own LDS.  16-byte units are stored at (unit ^ key of the
// row), so that the 16 rows of an operand are read from different banks.
template <bool kMX, bool kEven, int NT, int MT, int KW>
__global__ __launch_bounds__(64 * KW, 2) void wlinear_tile_kernel(WLinearArgs a) {
  constexpr int kBlock = kMX ? 32 : 16;
  constexpr int kTileN = 16 * NT, kTileM = 16 * MT;
  struct Lds {
    u32x4 w[NT][16][4];                        // [row][unit of 32 values]
    u32x4 x[MT][16][16];                       // [row][unit of 8 values]
    uint16_t s[NT][16][4];                     // [row][32 values]: their one or two scales
  };
  constexpr int kSums = NT * MT * 64 * sizeof(f32x4);
  constexpr int kBytes = sizeof(Lds) > kSums ? sizeof(Lds) : kSums;
  __shared__ __attribute__((aligned(16))) uint8_t mem[KW][kBytes];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  Lds& l = *reinterpret_cast<Lds*>(mem[wave]);
  // activation tiles of the same weight rows are neighbours
  const uint32_t tiles_m = (uint32_t)((a.M + kTileM - 1) / kTileM);
  const int64_t n0 = (int64_t)(blockIdx.x / tiles_m) * kTileN;
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * kTileM;
  const int K = (int)a.K, chunks = (K - 1) / kChunk + 1;   // K is below 2^31, K + 127 need not be
  const float t = kMX ? 1.0f : a.wt[0];
  const int rows_m = (int)min((int64_t)kTileM, a.M - m0);
  // loads in memory order: four lanes to a weight row, 16 to an activation row; rows past
  // N and M read the last row again
  const int wr = lane >> 2, wu = lane & 3, xr0 = lane >> 4, xu = lane & 15;
  const uint8_t* wp[NT];
  const uint8_t* sp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t row = min(n0 + 16 * n + wr, a.N - 1);
    wp[n] = a.wd + row * (K / 2) + 16 * wu;
    sp[n] = a.ws + row * (K / kBlock) + 32 / kBlock * wu;
  }
  const uint16_t* xp = a.x + m0 * a.x_stride + 8 * xu;

  f32x4 acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0, 0, 0, 0};

  // one chunk on its way; the registers are refilled as soon as it is staged
  u32x4 w[NT], x[4 * MT];
  uint32_t sb[NT];
  auto load = [&](int c) {
    const int left = K - c * kChunk;
    if (left >= kChunk) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // cached: a chunk of a row is half a line, another wave reads the other half (with
        // non-temporal loads 16.4 us instead of 12.7 at 61 x 4099 x 4112)
        w[n] = *reinterpret_cast<const u32x4_a8*>(wp[n] + c * (kChunk / 2));
        const uint8_t* s = sp[n] + c * (kChunk / kBlock);
        if constexpr (kMX) sb[n] = s[0];
        else if constexpr (kEven) sb[n] = *reinterpret_cast<const uint16_t*>(s);
        else sb[n] = s[0] | (uint32_t)s[1] << 8;
      }
#pragma unroll
      for (int m = 0; m < 4 * MT; ++m) {
        const int row = min(4 * m + xr0, rows_m - 1);
        x[m] = *reinterpret_cast<const u32x4*>(xp + row * a.x_stride + c * kChunk);
      }
    } else {
      // past K everything is zero (K % 16 == 0: a lane may hold half of its 32 weights)
      const bool half = 32 * wu + 16 <= left, full = 32 * wu + 32 <= left;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(wp[n] + c * (kChunk / 2));
        const uint8_t* s = sp[n] + c * (kChunk / kBlock);
        w[n] = u32x4{half ? p[0] : 0u, half ? p[1] : 0u, full ? p[2] : 0u, full ? p[3] : 0u};
        sb[n] = (half ? s[0] : 0u) | (!kMX && full ? (uint32_t)s[1] << 8 : 0u);
      }
#pragma unroll
      for (int m = 0; m < 4 * MT; ++m) {
        const int row = min(4 * m + xr0, rows_m - 1);
        x[m] = u32x4{0, 0, 0, 0};
        if (8 * xu < left)
          x[m] = *reinterpret_cast<const u32x4*>(xp + row * a.x_stride + c * kChunk);
      }
    }
  };
  auto stage = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l.w[n][wr][wu ^ (wr >> 2)] = w[n];
      l.s[n][wr][wu] = (uint16_t)sb[n];
    }
#pragma unroll
    for (int m = 0; m < 4 * MT; ++m) {
      const int row = 4 * (m & 3) + xr0;
      l.x[m >> 2][row][xu ^ row] = x[m];
    }
  };
  auto multiply = [&]() {
    u32x4 wf[NT];
    f32x2 sf[NT];                              // of the lane's first and last 16 values
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      wf[n] = l.w[n][r][q ^ (r >> 2)];
      sf[n] = scale_values<kMX>(l.s[n][r][q]);
    }
    // the reads of J steps are on their way before their first product (left alone, the
    // scheduler reads each operand right before its product and waits for it)
    constexpr int J = MT <= 2 ? 4 : 1;
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += J) {
      u32x4 xf[J][MT];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) xf[j][m] = l.x[m][r][(4 * q + j0 + j) ^ r];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const u32x4 e = dequant8<kMX>(wf[n][j0 + j], j0 + j < 2 ? sf[n].x : sf[n].y);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[n][m] = mfma(e, xf[j][m], acc[n][m]);
        }
    }
  };

  if (wave < chunks) load(wave);
  for (int c = wave; c < chunks; c += KW) {
    stage();
    if (c + KW < chunks) load(c + KW);
    multiply();
  }

  // join: rows n0 + 16 n + 4 q + i, column m0 + 16 m + r
  f32x4(*sums)[64] = reinterpret_cast<f32x4(*)[64]>(mem[wave]);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[n * MT + m][lane] = acc[n][m];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * MT * 64; i += 64 * KW) {
    const int tile = i >> 6, ln = i & 63;
    f32x4 v = reinterpret_cast<f32x4(*)[64]>(mem[0])[tile][ln];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += reinterpret_cast<f32x4(*)[64]>(mem[w])[tile][ln];
    const int64_t n = n0 + 16 * (tile / MT) + 4 * (ln >> 4), m = m0 + 16 * (tile % MT) + (ln & 15);
    if (m >= a.M) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (n + k >= a.N) break;
      float y = v[k] * t;
      if (a.bias) y += bf16_lo(a.bias[n + k]);
      const int64_t at = m * a.N + n + k;
      if (a.f32_out) static_cast<float*>(a.y)[at] = y;
      else static_cast<uint16_t*>(a.y)[at] = (uint16_t)pack_bf16x2(y, y);
    }
  }
}

// ---- few activation rows, or few weight rows --------------------------------------
// On the 4x4x4 instruction, 16 independent 4x4 products: a quad of lanes takes four weight
// rows (its columns) over the same 32 values of the inner dimension and four activation
// rows.  Each lane keeps the sums of its own weight row, so a block's scale multiplies the
// block's four sums instead of its 16 weights, and E2M1 enters as it is: about one VALU
// instruction per weight for up to four activation rows (a 16x16 tile takes two for any
// number, and its operands cross lanes).
//
// A wave takes 4 R weight rows (R to a lane) and walks the inner dimension 512 values at a
// time; the waves of a workgroup share its rows and split the inner dimension.  The
// activation comes in memory order and goes through the wave's own LDS.
constexpr int kQuadStep = 512;

// Sum over the lanes with the same lane % 4, in all of them.
__device__ __forceinline__ float sum_over_quads(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, true));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// kEven: scale rows start at even bytes (K % 32 == 0), so that a lane's two NVFP4 scales
// are one aligned load.  kMany: more than four activation rows, blockIdx.y counts the fours
// (apart, because what it takes in registers costs two rows a lane their fourth wave on a
// SIMD: 9.2 us instead of 7.8 at 1 x 4096 x 12288).
template <bool kMX, bool kEven, int R, int KW, bool kMany>
__global__ __launch_bounds__(64 * KW, R == 2 && !kMany ? 4 : 3) void wlinear_quad_kernel(WLinearArgs a) {
  constexpr int kBlock = kMX ? 32 : 16;
  constexpr int kRows = 4 * R;
  constexpr int U = R == 1 ? 4 : 2;     // steps in flight
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  __shared__ u32x4 xs[KW][4][64];
  __shared__ float sums[KW][kRows][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 3, g = lane >> 2;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int m0 = kMany ? 4 * (int)blockIdx.y : 0;
  const uint16_t* xp = a.x + m0 * a.x_stride;
  const int M = min((int)a.M - m0, 4);
  const int K = (int)a.K, steps = (K - 1) / kQuadStep + 1;   // K is below 2^31, K + 511 need not be
  const float t = kMX ? 1.0f : a.wt[0];
  const uint8_t* wp[R];
  const uint8_t* sp[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {         // rows past N read the last row again
    const int64_t row = min(n0 + 4 * j + i, a.N - 1);
    wp[j] = a.wd + row * (K / 2) + 16 * g;
    sp[j] = a.ws + row * (K / kBlock) + 32 / kBlock * g;
  }
  f32x4 acc[R];
#pragma unroll
  for (int j = 0; j < R; ++j) acc[j] = f32x4{0, 0, 0, 0};

  // The products of one step: w, sb the lane's weights and scales, x row m's unit `lane`.
  // Unit u of row m lies at u ^ (m % 4) in LDS: the four rows of a quad read from different
  // banks.  Rows past M are whatever LDS holds: they only reach sums that are not used.
  auto multiply = [&](const u32x4 (&w)[R], const uint32_t (&sb)[R], const u32x4 (&xr)[4]) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
      if (m < M) xs[wave][m][lane ^ (m & 3)] = xr[m];
    u32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = xs[wave][i][(4 * g + u) ^ i];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const f32x2 sf = scale_values<kMX>(sb[j]);
#pragma unroll
      for (int b = 0; b < 32 / kBlock; ++b) {
        f32x4 part = {0, 0, 0, 0};
#pragma unroll
        for (int u = b * kBlock / 8; u < (b + 1) * kBlock / 8; ++u) {   // 8 values each
          const u32x4 e = dequant8<true>(w[j][u], 1.0f);
          part = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(
              __builtin_bit_cast(s16x4, u32x2{x[u].x, x[u].y}),
              __builtin_bit_cast(s16x4, u32x2{e.x, e.y}), part, 0, 0, 0);
          part = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(
              __builtin_bit_cast(s16x4, u32x2{x[u].z, x[u].w}),
              __builtin_bit_cast(s16x4, u32x2{e.z, e.w}), part, 0, 0, 0);
        }
        const float d = b ? sf.y : sf.x;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][c] = __builtin_fmaf(part[c], d, acc[j][c]);
      }
    }
  };

  auto load = [&](int s, u32x4 (&w)[R], uint32_t (&sb)[R], u32x4 (&xr)[4]) {
    const int left = K - s * kQuadStep;
    if (left >= kQuadStep) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        w[j] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_a8*>(wp[j] + s * (kQuadStep / 2)));
        const uint8_t* q = sp[j] + s * (kQuadStep / kBlock);
        if constexpr (kMX) sb[j] = q[0];
        else if constexpr (kEven) sb[j] = *reinterpret_cast<const uint16_t*>(q);
        else sb[j] = q[0] | (uint32_t)q[1] << 8;
      }
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (m < M) xr[m] = reinterpret_cast<const u32x4*>(xp + m * a.x_stride + s * kQuadStep)[lane];
    } else {
      // past K everything is zero (K % 16 == 0: a lane may hold half of its 32 weights)
      const bool half = 32 * g + 16 <= left, full = 32 * g + 32 <= left;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(wp[j] + s * (kQuadStep / 2));
        const uint8_t* q = sp[j] + s * (kQuadStep / kBlock);
        w[j] = u32x4{half ? p[0] : 0u, half ? p[1] : 0u, full ? p[2] : 0u, full ? p[3] : 0u};
        sb[j] = (half ? q[0] : 0u) | (!kMX && full ? (uint32_t)q[1] << 8 : 0u);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        xr[m] = u32x4{0, 0, 0, 0};
        if (m < M && 8 * lane < left)
          xr[m] = reinterpret_cast<const u32x4*>(xp + m * a.x_stride + s * kQuadStep)[lane];
      }
    }
  };
  for (int s = wave; s < steps; s += KW * U) {
    u32x4 w[U][R], xr[U][4];
    uint32_t sb[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + KW * u < steps) load(s + KW * u, w[u], sb[u], xr[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + KW * u < steps) multiply(w[u], sb[u], xr[u]);
  }

#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = sum_over_quads(acc[j][c]);
      if (g == 0) sums[wave][4 * j + i][c] = v;
    }
  __syncthreads();
  for (int e = threadIdx.x; e < kRows * M; e += 64 * KW) {
    const int n = e % kRows, m = e / kRows;
    if (n0 + n >= a.N) continue;
    float v = sums[0][n][m];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += sums[w][n][m];
    v *= t;
    if (a.bias) v += bf16_lo(a.bias[n0 + n]);
    const int64_t at = (int64_t)(m0 + m) * a.N + n0 + n;
    if (a.f32_out) static_cast<float*>(a.y)[at] = v;
    else static_cast<uint16_t*>(a.y)[at] = (uint16_t)pack_bf16x2(v, v);
  }
}

// Kernel and tile for a shape: 16 NT weight rows by 16 MT activation rows (MT 0: the quad
// kernel with R = NT), KW waves.
struct Shape {
  int nt, mt, kw;
};
int64_t tiles_of(const WLinearArgs& a, const Shape& h);

// The quad kernel wherever its workgroups of 4 or 8 weight rows by 4 activation rows fit on
// the GPU one to a CU: fewer rows a lane are more workgroups, each with a shorter chain (1 x
// 256 x 256: 2.8 us, with 16 weight rows 3.7; 1 x 1024 x 8192: 4.0 and 6.3; 3 x 1073 x 11344: 6.3
// and 8.9; 16 x 256 x 8192: 4.1, a tile 6.9; but two to a CU, 16 x 1024 x 4096: 6.5, a tile
// 4.9).  Then for up to 4 activation rows, or 2 where the weight rows alone give two tiles
// per CU (4 x 4096 x 12288: 9.3, a tile 9.6; 4 x 12288 x 4096: 9.1, a tile 8.5); one
// activation row is little enough to be read by twice the workgroups (1 x 4096 x 12288: 7.8
// with 8 weight rows, 8.2 with 16; 2 x 4096 x 12288: 9.2 and 8.5).
//
// Otherwise the tile that is done first, by what one workgroup of each takes at K = 4096 (us,
// measured) times the rounds of 256 workgroups.  Eight waves on 32 activation rows take most
// of a CU's LDS: no other workgroup runs beside them, so they are for one round (61 x 4099 x
// 4096: 10.2 us, four waves 11.0; 24 x 8192 x 4096: 8.4 and 9.0; but two rounds, 64 x 16384 x
// 1024: 15.1 and 9.9).
Shape shape_of(const WLinearArgs& a) {
  const Shape few[] = {{1, 0, 8}, {2, 0, 8}};
  for (const Shape& h : few)
    if (tiles_of(a, h) <= kCUs) return h;
  const bool wide = a.N >= 2 * 16 * kCUs;
  if (a.M <= (wide ? 2 : 4)) return wide ? Shape{4, 0, 4} : Shape{a.M == 1 ? 2 : 4, 0, 8};
  constexpr struct {
    Shape shape;
    float us;
  } kTiles[] = {{{1, 1, 8}, 2.6f}, {{2, 1, 8}, 4.0f}, {{3, 1, 8}, 6.2f},
                {{2, 2, 8}, 6.2f}, {{2, 2, 4}, 6.6f}, {{3, 2, 8}, 8.5f},
                {{3, 2, 4}, 9.0f}, {{3, 4, 4}, 14.7f}};
  Shape best = kTiles[0].shape;
  float least = INFINITY;
  for (const auto& c : kTiles) {
    const int64_t rounds = (tiles_of(a, c.shape) + kCUs - 1) / kCUs;
    if (c.shape.mt == 2 && c.shape.kw == 8 && rounds > 1) continue;
    const float us = c.us * (float)rounds;
    if (us < least) {
      least = us;
      best = c.shape;
    }
  }
  return best;
}
int64_t tiles_of(const WLinearArgs& a, const Shape& h) {
  if (h.mt == 0) return ((a.N + 4 * h.nt - 1) / (4 * h.nt)) * ((a.M + 3) / 4);
  return ((a.N + 16 * h.nt - 1) / (16 * h.nt)) * ((a.M + 16 * h.mt - 1) / (16 * h.mt));
}

template <int NT, int MT, int KW>
bool launch_if(const WLinearArgs& a, const Shape& h, hipStream_t s) {
  if (h.nt != NT || h.mt != MT || h.kw != KW) return false;
  const uint32_t grid = (uint32_t)tiles_of(a, h);
  if (a.mx) wlinear_tile_kernel<true, true, NT, MT, KW><<<grid, 64 * KW, 0, s>>>(a);
  else if (a.K % 32 == 0) wlinear_tile_kernel<false, true, NT, MT, KW><<<grid, 64 * KW, 0, s>>>(a);
  else wlinear_tile_kernel<false, false, NT, MT, KW><<<grid, 64 * KW, 0, s>>>(a);
  return true;
}

template <int R, int KW, bool kMany>
bool launch_quad_if(const WLinearArgs& a, const Shape& h, hipStream_t s) {
  if (h.nt != R || h.mt != 0 || h.kw != KW || (a.M > 4) != kMany) return false;
  const dim3 grid((uint32_t)((a.N + 4 * R - 1) / (4 * R)), (uint32_t)((a.M + 3) / 4));
  if (a.mx) wlinear_quad_kernel<true, true, R, KW, kMany><<<grid, 64 * KW, 0, s>>>(a);
  else if (a.K % 32 == 0) wlinear_quad_kernel<false, true, R, KW, kMany><<<grid, 64 * KW, 0, s>>>(a);
  else wlinear_quad_kernel<false, false, R, KW, kMany><<<grid, 64 * KW, 0, s>>>(a);
  return true;
}

}  // namespace

int64_t wlinear_threads(const WLinearArgs& a) {
  const Shape h = shape_of(a);
  return tiles_of(a, h) * 64 * h.kw;
}

hipError_t launch_wlinear(const WLinearArgs& a, hipStream_t s) {
  const Shape h = shape_of(a);
  const bool launched =
      launch_quad_if<1, 8, false>(a, h, s) || launch_quad_if<2, 8, false>(a, h, s) ||
      launch_quad_if<4, 8, false>(a, h, s) || launch_quad_if<4, 4, false>(a, h, s) ||
      launch_quad_if<1, 8, true>(a, h, s) || launch_quad_if<2, 8, true>(a, h, s) ||
      launch_if<1, 1, 8>(a, h, s) ||
      launch_if<2, 1, 8>(a, h, s) || launch_if<3, 1, 8>(a, h, s) || launch_if<2, 2, 8>(a, h, s) ||
      launch_if<2, 2, 4>(a, h, s) || launch_if<3, 2, 8>(a, h, s) || launch_if<3, 2, 4>(a, h, s) ||
      launch_if<3, 4, 4>(a, h, s);
  if (!launched) return hipErrorInvalidConfiguration;
  return hipGetLastError();
}

}  // namespace fos
