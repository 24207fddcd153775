// Weight-only quantized linear layer: bf16 activations times a 4-bit weight record,
//   y[m][n] = t * sum_k x[m][k] E(w[n][k]) D(s[n][k / block]) + bias[n].
// The weight is read once; its bytes bound the call (x and y are small beside it).
//
// Matrix form, on the 16x16x32 bf16 instruction: A = 16 weight rows, B = 16 activation
// rows, so a weight is converted to bf16 once for up to 64 activation rows.  E2M1 x E4M3
// has at most 6 significant bits and E2M1 x 2^e two: both are exact in bf16, products
// are exact in fp32, and every sum is fp32.  y is rounded once.
//
// A wave walks the inner dimension in chunks of 128.  For each weight row (r = lane % 16)
// its four lanes (q = lane / 16) read 16 contiguous bytes each, and exchange them so that
// in step j lane q holds the values k = 32 j + 8 q .. + 7: then the activation's loads
// are 64 contiguous bytes per row as well.  The waves of a workgroup share its output
// tile and split the inner dimension; they join in LDS in a fixed order.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kChunk = 128;   // values of the inner dimension per wave and step

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Weight rows are K / 2 bytes apart: 8-byte alignment (K % 16 == 0), scales any.
typedef uint32_t u32x4_a8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
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
template <bool kMX>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return kMX ? __uint_as_float(byte << 23) : e4m3_decode(byte & 0x7fu);
}

// One chunk of one weight row as its four lanes load it: word j of lane q is 16 q + 4 j
// bytes into the chunk.
template <bool kMX>
struct RawW {
  u32x4 w;
  u32x2 s;      // NVFP4: the chunk's 8 block scales; MXFP4: its 4 in s.x
};

// 4x4 exchange of words between the lanes q = 0..3 of a row: word j of lane q becomes
// word q of lane j.
__device__ __forceinline__ u32x4 exchange(u32x4 w) {
  auto a = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

template <bool kMX, int NT, int MT, int KW>
__global__ __launch_bounds__(64 * KW) void wlinear_kernel(WLinearArgs a) {
  // chunks in flight per wave: their x must fit the registers too
  constexpr int U = MT == 1 ? (KW > 8 ? 2 : 4) : MT == 2 ? 2 : 1;
  constexpr int kBlock = kMX ? 32 : 16;
  constexpr int kTileN = 16 * NT, kTileM = 16 * MT;
  __shared__ f32x4 sums[KW][NT * MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  // activation tiles of the same weight rows are neighbours
  const uint32_t tiles_m = (uint32_t)((a.M + kTileM - 1) / kTileM);
  const int64_t n0 = (int64_t)(blockIdx.x / tiles_m) * kTileN;
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * kTileM;
  const int chunks = (int)(a.K / kChunk);      // whole ones
  const uint8_t* wp[NT];
  const uint8_t* sp[NT];
  const uint16_t* xp[MT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {               // rows past N read the last row again
    const int64_t row = min(n0 + 16 * n + r, a.N - 1);
    wp[n] = a.wd + row * (a.K / 2);
    sp[n] = a.ws + row * (a.K / kBlock);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) xp[m] = a.x + min(m0 + 16 * m + r, a.M - 1) * a.x_stride + 8 * q;

  f32x4 acc[NT][MT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0, 0, 0, 0};

  RawW<kMX> raw[U][NT];
  auto load_w = [&](int c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = min(c + KW * u, chunks - 1);      // past the end: not used
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        raw[u][n].w = *reinterpret_cast<const u32x4_a8*>(wp[n] + (int64_t)cu * (kChunk / 2) + 16 * q);
        const uint8_t* s = sp[n] + (int64_t)cu * (kChunk / kBlock);
        if constexpr (kMX) raw[u][n].s.x = *reinterpret_cast<const u32_a1*>(s);
        else raw[u][n].s = *reinterpret_cast<const u32x2_a1*>(s);
      }
    }
  };
  if (wave < chunks) load_w(wave);
  for (int c = wave; c < chunks; c += KW * U) {
    u32x4 xf[U][MT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = min(c + KW * u, chunks - 1);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xf[u][m][j] = *reinterpret_cast<const u32x4*>(xp[m] + (int64_t)cu * kChunk + 32 * j);
    }
    RawW<kMX> cur[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) cur[u][n] = raw[u][n];
    if (c + KW * U < chunks) load_w(c + KW * U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + KW * u >= chunks) break;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4 w = exchange(cur[u][n].w);
        // block scales of this lane's steps: NVFP4 byte 2 j + q / 2, MXFP4 byte j
        const uint32_t s0 = kMX ? cur[u][n].s.x : cur[u][n].s.x >> (8 * (q >> 1));
        const uint32_t s1 = kMX ? cur[u][n].s.x >> 16 : cur[u][n].s.y >> (8 * (q >> 1));
        const uint32_t sb[4] = {s0 & 0xff, (kMX ? s0 >> 8 : s0 >> 16) & 0xff, s1 & 0xff,
                                (kMX ? s1 >> 8 : s1 >> 16) & 0xff};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 wf = dequant8<kMX>(w[j], scale_value<kMX>(sb[j]));
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[n][m] = mfma(wf, xf[u][m][j], acc[n][m]);
        }
      }
    }
  }
  // the last K % 128 values, in the layout of the steps; what lies past K is zero
  if (chunks % KW == wave && a.K % kChunk) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = (int64_t)chunks * kChunk + 32 * j + 8 * q;
      const bool in = k < a.K;
      u32x4 xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
        xf[m] = in ? *reinterpret_cast<const u32x4*>(xp[m] + (k - 8 * q)) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t w = in ? *reinterpret_cast<const uint32_t*>(wp[n] + k / 2) : 0u;
        const uint32_t s = in ? sp[n][k / kBlock] : 0u;
        const u32x4 wf = dequant8<kMX>(w, scale_value<kMX>(s));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = mfma(wf, xf[m], acc[n][m]);
      }
    }
  }

  // join: rows n0 + 16 n + 4 q + i, column m0 + 16 m + r
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[wave][n * MT + m][lane] = acc[n][m];
  __syncthreads();
  const float t = kMX ? 1.0f : a.wt[0];
  for (int i = threadIdx.x; i < NT * MT * 64; i += 64 * KW) {
    const int tile = i >> 6, l = i & 63;
    f32x4 v = sums[0][tile][l];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += sums[w][tile][l];
    const int64_t n = n0 + 16 * (tile / MT) + 4 * (l >> 4), m = m0 + 16 * (tile % MT) + (l & 15);
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

// Tile and split for a shape: 16 NT weight rows, 16 MT activation rows, KW waves.
struct Shape {
  int nt, mt, kw;
};
Shape shape_of(const WLinearArgs& a) {
  const bool few = a.N < 16 * 512;             // weight rows for fewer than 512 workgroups of 16
  if (a.M <= 16) return few ? Shape{1, 1, 16} : Shape{1, 1, 4};
  if (a.M <= 32) return few ? Shape{1, 2, 8} : Shape{2, 2, 4};
  return few ? Shape{1, 4, 8} : Shape{2, 4, 4};
}
int64_t tiles_of(const WLinearArgs& a, const Shape& h) {
  return ((a.N + 16 * h.nt - 1) / (16 * h.nt)) * ((a.M + 16 * h.mt - 1) / (16 * h.mt));
}

template <int NT, int MT, int KW>
bool launch_if(const WLinearArgs& a, const Shape& h, hipStream_t s) {
  if (h.nt != NT || h.mt != MT || h.kw != KW) return false;
  const uint32_t grid = (uint32_t)tiles_of(a, h);
  if (a.mx) wlinear_kernel<true, NT, MT, KW><<<grid, 64 * KW, 0, s>>>(a);
  else wlinear_kernel<false, NT, MT, KW><<<grid, 64 * KW, 0, s>>>(a);
  return true;
}

}  // namespace

int64_t wlinear_threads(const WLinearArgs& a) {
  const Shape h = shape_of(a);
  return tiles_of(a, h) * 64 * h.kw;
}

hipError_t launch_wlinear(const WLinearArgs& a, hipStream_t s) {
  const Shape h = shape_of(a);
  (void)(launch_if<1, 1, 16>(a, h, s) || launch_if<1, 1, 4>(a, h, s) ||
         launch_if<1, 2, 8>(a, h, s) || launch_if<2, 2, 4>(a, h, s) ||
         launch_if<1, 4, 8>(a, h, s) || launch_if<2, 4, 4>(a, h, s));
  return hipGetLastError();
}

}  // namespace fos
