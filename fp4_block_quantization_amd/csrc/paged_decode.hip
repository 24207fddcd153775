// Attention of one new token per sequence over a paged key-value cache.  For sequence b
// and query head h (kv head h / G), over the visible tokens j (below the length, inside
// the window, in a page that the cache holds):
//   s_j = scale * q . k_j,   lse = log sum exp s_j,   out = sum exp(s_j - lse) v_j,
// in one pass over K and V with the running maximum m and sum l of the softmax:
//   m' = max(m, s),  l' = l exp(m - m') + exp(s - m'),  o' = o exp(m - m') + exp(s - m') v.
// Statistics and sums are fp32; out is rounded once.
//
// Matrix form.  One wave takes 32 tokens at a time for up to 16 query heads of one kv
// head (fewer heads leave columns of zeros: the kernel reads K and V once whatever G is,
// and the matrix cores have the rate to spare).  Both products put the heads on the
// columns of the 16x16x32 instruction:
//   S^T [token][head] = K Q^T    A operand: 16 K rows, straight from memory
//   O^T [d][head]     = V^T P^T  A operand: V, 8 tokens x 8 d of a lane transposed in
//                                registers (one v_perm_b32 for two values)
// A lane of group q = lane / 16 supplies the K rows r = lane % 16 as tokens
// 8 (r / 4) + 4 u + r % 4 (u = 0, 1: two instructions), so that its results, rows
// 4 q + i of S^T, are the tokens 8 q + 4 u + i: exactly the 8 tokens that the lane's
// group supplies to the second product.  The weights go from one product into the
// other without leaving their lane, and the running statistics of a head are per lane.
//
// Split.  Every workgroup takes one chunk of one sequence's tokens for one kv head.  The
// chunk length is set on the device from the lengths themselves (all tokens over the
// wanted number of workgroups), so that ragged batches stay balanced and the host needs
// no length.  A sequence of several chunks leaves partial (m, l, o) that a second kernel
// joins; the order of every sum depends on the lengths alone.
#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kHeads = 16;            // query heads per workgroup: columns of the products
constexpr int kTargetItems = 1024;    // chunks wanted over the whole batch
constexpr int kMinChunk = 512;        // tokens of a chunk, at least
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

struct Plan {
  DecodeArgs a;
  int groups;              // workgroups' worth of query heads per kv head: ceil(G / 16)
  int rows;                // query heads of a partial: min(G, 16)
  // x / d = (x * page_magic) >> 36 for d = page_size / 8 (at most 512) and x < 2^27:
  // page_magic = ceil(2^36 / d) is too large by less than 1, x * (less than d) < 2^36
  uint64_t page_magic;
};

// Partial results: per chunk m[rows], l[rows], o[rows][dim].
__device__ __forceinline__ int64_t part_stride(const Plan& p) {
  return (int64_t)p.rows * (p.a.c.dim + 2);
}

// ---- chunks ----------------------------------------------------------------------
// Visible range of a sequence: tokens [first, last), tiles counted from `base`, first
// rounded down to a group of 8 tokens.
struct Range {
  int base, first, last;
};
__device__ __forceinline__ Range range_of(const Plan& p, int len) {
  const int64_t w = p.a.window;
  const int first = (w > 0 && w < len) ? len - (int)w : 0;
  const int last = min(len, p.a.pages_per_seq * p.a.c.page_size);
  if (first >= last) return Range{0, 0, 0};
  return Range{first & ~7, first, last};
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Tokens per chunk, a multiple of `step`: enough that the batch gives about kTargetItems.
__device__ __forceinline__ int chunk_tokens(const Plan& p, int lane, int step) {
  int64_t total = 0;
  for (int b = lane; b < p.a.B; b += 64) {
    const Range r = range_of(p, p.a.lens[b]);
    total += r.last - r.base;
  }
  total = wave_sum(total) * (p.a.c.heads * p.groups);
  int64_t c = (total + kTargetItems - 1) / kTargetItems;
  c = max(c, (int64_t)kMinChunk);
  c = (c + step - 1) / step * step;
  return (int)min(c, (int64_t)1 << 30);
}

__device__ __forceinline__ int chunks_of(const Range& r, int chunk) {
  return max(1, (r.last - r.base + chunk - 1) / chunk);   // an empty sequence writes its zeros
}

// Sequence and chunk-and-head number of work item i, or b = -1 past the last.  Every lane
// of the wave gets the same answer.
struct Item {
  int b, in_b, first_item;
};
__device__ __forceinline__ Item find_item(const Plan& p, int lane, int chunk, int i) {
  const int per = p.a.c.heads * p.groups;
  int before = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 64) {
    const int b = b0 + lane;
    const int n = b < p.a.B ? chunks_of(range_of(p, p.a.lens[b]), chunk) * per : 0;
    int upto = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int up = __shfl_up(upto, off);
      if (lane >= off) upto += up;
    }
    const int start = before + upto - n;
    const uint64_t hit = __ballot(i >= start && i < start + n);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int s = __shfl(start, l);
      return Item{b0 + l, i - s, s};
    }
    before += __shfl(upto, 63);
  }
  return Item{-1, 0, 0};
}

// ---- one wave's pieces -------------------------------------------------------------
// The dim of a row in pieces of 128, 64 and 32 values: in a piece of P a lane holds
// P / 16 consecutive values of each V row (r = lane % 16: values P / 16 r ..), and of an
// NVFP4 K row P / 4 consecutive ones (group q).
template <int D>
struct Pieces {
  static constexpr int n128 = D / 128, n64 = (D % 128) / 64, n32 = (D % 64) / 32;
  static constexpr int count = n128 + n64 + n32;
  static constexpr int size(int i) { return i < n128 ? 128 : i < n128 + n64 ? 64 : 32; }
  static constexpr int at(int i) {
    return i <= n128 ? 128 * i : 128 * n128 + (i > n128 && n64 ? 64 : 0) +
           (i > n128 + n64 ? 32 * (i - n128 - n64) : 0);
  }
};

__device__ __forceinline__ float max_over_groups(float v) {   // lanes l, l+16, l+32, l+48
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Eight nibbles times one block scale as eight halves: E2M1 x E4M3 has at most 6
// significant bits between 2^-10 and 2688, so it is exact in half precision.
__device__ __forceinline__ f16x2 e4m3_pair(uint32_t byte) {
  const f16x2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(byte, 1.0f, false);
  return f16x2{s.x, s.x};
}
__device__ __forceinline__ u32x4 dequant8(uint32_t w, f16x2 s) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
               __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

template <bool kNVFP4>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kNVFP4)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// Cache row of the first token of a group of 8 (a group never crosses a page), or -1.
__device__ __forceinline__ int64_t group_row(const Plan& p, const int32_t* table, int head, int tok) {
  const uint32_t g = (uint32_t)tok >> 3;
  const int page = (int)((g * p.page_magic) >> 36);
  if (page >= p.a.pages_per_seq) return -1;
  const int id = table[page];
  if (id < 0 || id >= p.a.c.num_pages) return -1;
  return ((int64_t)id * p.a.c.heads + head) * p.a.c.page_size + (tok - page * p.a.c.page_size);
}

template <bool kNVFP4, int D>
__global__ __launch_bounds__(kThreads) void paged_decode_kernel(Plan p) {
  constexpr int kSteps = D / 32;               // 32-value steps of the first product
  constexpr int kTiles = D / 16;               // 16-row tiles of the second
  constexpr int kPad = D + 4;
  using P = Pieces<D>;
  __shared__ __attribute__((aligned(16))) float so[kWaves][kHeads][kPad];
  __shared__ float sm[kWaves][kHeads], sl[kWaves][kHeads];
  const DecodeArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int chunk = chunk_tokens(p, lane, 32 * kWaves);
  const Item it = find_item(p, lane, chunk, blockIdx.x);
  if (it.b < 0) return;
  const int per = a.c.heads * p.groups;
  const int ci = it.in_b / per, hg = it.in_b % per;
  const int head = hg / p.groups, g0 = (hg % p.groups) * kHeads;
  const int rows = min(kHeads, a.G - g0);
  const Range rg = range_of(p, a.lens[it.b]);
  const int begin = rg.base + ci * chunk, end = min(rg.last, begin + chunk);
  const int32_t* table = a.table + it.b * a.table_stride;

  // Queries: column r of both products, scaled by a power of two so that the largest is in
  // [1, 2): exact in bf16, and in half precision but for values below 2^-14 of it, which
  // keep an absolute 2^-25 of the largest.  The power goes into the scale of the scores.
  const uint16_t* qrow = a.q + it.b * a.q_stride + (int64_t)(head * a.G + g0 + r) * D;
  u32x4 qf[kSteps];
  float cs;
  {
    u32x4 raw[kSteps];
    uint32_t mx = 0;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      int d = 32 * j + 8 * q;                  // the 8 values of this lane in step j
      if (kNVFP4) {
#pragma unroll
        for (int i = 0; i < P::count; ++i)
          if (32 * j >= P::at(i) && 32 * j < P::at(i) + P::size(i))
            d = P::at(i) + P::size(i) / 4 * q + (32 * j - P::at(i)) / 4;
      }
      raw[j] = r < rows ? *reinterpret_cast<const u32x4*>(qrow + d) : u32x4{0, 0, 0, 0};
      mx = pk_max_abs4(mx, make_uint4(raw[j].x, raw[j].y, raw[j].z, raw[j].w));
    }
    const float top = max_over_groups(__uint_as_float(pk_max_to_f32_bits(mx)));
    const int e = top > 0.0f ? ilogbf(top) : 0;
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = ldexpf(bf16_lo(raw[j][i]), -e), y = ldexpf(bf16_hi(raw[j][i]), -e);
        qf[j][i] = kNVFP4 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
      }
    cs = ldexpf(a.scale * kLog2e * (kNVFP4 ? a.c.kt[0] : 1.0f), e);
  }

  f32x4 o[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) o[i] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;

  for (int t0 = begin + 32 * wave; t0 < end; t0 += 32 * kWaves) {
    // rows of this lane's K tokens and V tokens; lanes of an absent page read row 0 (of a
    // cache with at least one page) and are masked
    const int gk = t0 + 8 * (r >> 2), gv = t0 + 8 * q;
    const int64_t rk = gk < end ? group_row(p, table, head, gk) : -1;
    const int64_t rv = gv < end ? group_row(p, table, head, gv) : -1;
    const int64_t krow = rk < 0 ? 0 : rk + (r & 3), vrow = max(rv, (int64_t)0);
    f32x4 s[2];
    u32x4 vt[kTiles];                          // V^T: tile i, tokens 8 q .. 8 q + 7
    uint32_t seen = 0;                         // bit e: token gv + e is visible
#pragma unroll
    for (int e = 0; e < 8; ++e) seen |= (uint32_t)(rv >= 0 && gv + e >= rg.first && gv + e < end) << e;
    const bool all = __all(seen == 0xffu);
    if constexpr (kNVFP4) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* kp = a.c.k + (krow + 4 * u) * (D / 2);
        const uint8_t* sp = a.c.ks + (krow + 4 * u) * (D / 16);
        s[u] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < P::count; ++i) {
          constexpr int kN[3] = {4, 2, 1};
          const int n = P::size(i) == 128 ? kN[0] : P::size(i) == 64 ? kN[1] : kN[2];
          const uint32_t* w = reinterpret_cast<const uint32_t*>(kp + P::at(i) / 2 + P::size(i) / 8 * q);
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const int d = P::at(i) + P::size(i) / 4 * q + 8 * j;
            s[u] = mfma<true>(dequant8(w[j], e4m3_pair(sp[d / 16])), qf[P::at(i) / 32 + j], s[u]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < P::count; ++i) {
        const int per16 = P::size(i) / 16;     // values of a lane and row: 8, 4 or 2
        uint32_t h[8][4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t row = vrow + e;
          const int d = P::at(i) + per16 * r;
          const uint8_t* w = a.c.v + row * (D / 2) + d / 2;
          uint32_t sb = a.c.vs[row * (D / 16) + d / 16];
          if (!all && !((seen >> e) & 1)) sb = 0;
          const f16x2 sc = e4m3_pair(sb);
          const uint32_t word = per16 == 8 ? *reinterpret_cast<const uint32_t*>(w)
                                : per16 == 4 ? *reinterpret_cast<const uint16_t*>(w) : *w;
          const u32x4 x = dequant8(word, sc);
          h[e][0] = x.x; h[e][1] = x.y; h[e][2] = x.z; h[e][3] = x.w;
        }
#pragma unroll
        for (int c = 0; c < per16 / 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            vt[P::at(i) / 16 + 2 * c][e] = __builtin_amdgcn_perm(h[2 * e + 1][c], h[2 * e][c], 0x05040100u);
            vt[P::at(i) / 16 + 2 * c + 1][e] = __builtin_amdgcn_perm(h[2 * e + 1][c], h[2 * e][c], 0x07060302u);
          }
      }
    } else {
      const uint16_t* kb = reinterpret_cast<const uint16_t*>(a.c.k);
      const uint16_t* vb = reinterpret_cast<const uint16_t*>(a.c.v);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint16_t* kp = kb + (krow + 4 * u) * D + 8 * q;
        s[u] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
          s[u] = mfma<false>(*reinterpret_cast<const u32x4*>(kp + 32 * j), qf[j], s[u]);
      }
#pragma unroll
      for (int i = 0; i < P::count; ++i) {
        const int per16 = P::size(i) / 16;
        uint32_t h[8][4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t* w = vb + (vrow + e) * D + P::at(i) + per16 * r;
          if (per16 == 8) {
            const u32x4 x = *reinterpret_cast<const u32x4*>(w);
            h[e][0] = x.x; h[e][1] = x.y; h[e][2] = x.z; h[e][3] = x.w;
          } else if (per16 == 4) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(w);
            h[e][0] = x.x; h[e][1] = x.y;
          } else {
            h[e][0] = *reinterpret_cast<const uint32_t*>(w);
          }
        }
        if (!all) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int c = 0; c < per16 / 2; ++c) h[e][c] = (seen >> e) & 1 ? h[e][c] : 0u;
        }
#pragma unroll
        for (int c = 0; c < per16 / 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            vt[P::at(i) / 16 + 2 * c][e] = __builtin_amdgcn_perm(h[2 * e + 1][c], h[2 * e][c], 0x05040100u);
            vt[P::at(i) / 16 + 2 * c + 1][e] = __builtin_amdgcn_perm(h[2 * e + 1][c], h[2 * e][c], 0x07060302u);
          }
      }
    }

    // scores in powers of two, masked; running maximum and weights
    float w[8], top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = s[e >> 2][e & 3] * cs;
      if (!all && !((seen >> e) & 1)) w[e] = -INFINITY;
      top = fmaxf(top, w[e]);
    }
    top = max_over_groups(top);
    if (__any(top > m)) {
      const float m2 = fmaxf(m, top);
      const float f = m2 == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[i] *= f;
    }
    const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = __builtin_amdgcn_exp2f(w[e] - m0);
      l += w[e];
    }
    // weights of the second product: half precision (11 bits) beside exact half-precision
    // V; beside bf16 V as the sum of two bf16 (16 bits), since one would round the weights
    // to 8 bits
    u32x4 hi;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      hi[e] = kNVFP4 ? pack_f16x2(w[2 * e], w[2 * e + 1]) : pack_bf16x2(w[2 * e], w[2 * e + 1]);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[i] = mfma<kNVFP4>(vt[i], hi, o[i]);
    if constexpr (!kNVFP4) {
      u32x4 lo;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        lo[e] = pack_bf16x2(w[2 * e] - bf16_lo(hi[e]), w[2 * e + 1] - bf16_hi(hi[e]));
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[i] = mfma<false>(vt[i], lo, o[i]);
    }
  }

  // join the waves
  l = sum_over_groups(l);
  if (q == 0) {
    sm[wave][r] = m;
    sl[wave][r] = l;
  }
  if (r < rows) {
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int per16 = P::size(i) / 16;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < per16; ++k)
          so[wave][r][P::at(i) + per16 * (4 * q + c) + k] = o[P::at(i) / 16 + k][c];
    }
  }
  __syncthreads();
  const bool whole = chunks_of(rg, chunk) == 1;
  const float vt0 = kNVFP4 ? a.c.vt[0] : 1.0f;
  float* part = static_cast<float*>(a.ws) + (int64_t)blockIdx.x * part_stride(p);
  for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
    const int g = i / (D / 2), d = 2 * (i % (D / 2));
    float mm = sm[0][g];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sm[w][g]);
    float ll = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = sm[w][g] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sm[w][g] - mm);
      ll += f * sl[w][g];
      x += f * so[w][g][d];
      y += f * so[w][g][d + 1];
    }
    const int64_t hrow = (int64_t)it.b * a.Hq + head * a.G + g0 + g;
    if (whole) {
      const float n = ll > 0.0f ? vt0 / ll : 0.0f;
      *reinterpret_cast<uint32_t*>(a.out + hrow * D + d) = pack_bf16x2(x * n, y * n);
      if (d == 0 && a.lse) a.lse[hrow] = ll > 0.0f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    } else {
      *reinterpret_cast<float2*>(part + 2 * p.rows + g * D + d) = make_float2(x, y);
      if (d == 0) {
        part[g] = mm;
        part[p.rows + g] = ll;
      }
    }
  }
}

// One workgroup per sequence and query head: joins the partials of its chunks.
__global__ __launch_bounds__(kThreads) void join_kernel(Plan p) {
  __shared__ float so[kThreads][4];
  __shared__ float sl[kThreads];
  const DecodeArgs& a = p.a;
  const int lane = threadIdx.x & 63;
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  const int chunk = chunk_tokens(p, lane, 32 * kWaves);
  const int n = chunks_of(range_of(p, a.lens[b]), chunk);
  if (n == 1) return;
  const int per = a.c.heads * p.groups;
  int64_t before = 0;
  for (int i = lane; i < b; i += 64) before += chunks_of(range_of(p, a.lens[i]), chunk);
  before = wave_sum(before) * per;
  const int hk = h / a.G, g = h % a.G, hg = hk * p.groups + g / kHeads, row = g % kHeads;
  const float* part = static_cast<const float*>(a.ws) + (before + hg) * part_stride(p);
  const int64_t step = per * part_stride(p);        // from chunk to chunk
  const int D = a.c.dim, quads = D / 4;              // threads of one partial: 8 to 64
  const int slots = kThreads / quads, t = threadIdx.x % quads, slot = threadIdx.x / quads;
  float m = -INFINITY;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, part[i * step + row]);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  float l = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  if (slot < slots && m > -INFINITY) {
    for (int i = slot; i < n; i += slots) {
      const float mi = part[i * step + row];
      const float f = __builtin_amdgcn_exp2f(mi - m);   // 0 for a chunk that saw nothing
      l += f * part[i * step + p.rows + row];
      const float2* src = reinterpret_cast<const float2*>(part + i * step + 2 * p.rows + row * D + 4 * t);
      const float2 x = src[0], y = src[1];
      o += f * f32x4{x.x, x.y, y.x, y.y};
    }
  }
  sl[threadIdx.x] = l;
#pragma unroll
  for (int k = 0; k < 4; ++k) so[threadIdx.x][k] = o[k];
  __syncthreads();
  if (slot != 0) return;
  for (int s = 1; s < slots; ++s) {
    l += sl[s * quads + t];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] += so[s * quads + t][k];
  }
  const float v = l > 0.0f ? (a.c.nvfp4 ? a.c.vt[0] : 1.0f) / l : 0.0f;
  const int64_t hrow = (int64_t)b * a.Hq + h;
  *reinterpret_cast<u32x2*>(a.out + hrow * D + 4 * t) =
      u32x2{pack_bf16x2(o[0] * v, o[1] * v), pack_bf16x2(o[2] * v, o[3] * v)};
  if (t == 0 && a.lse) a.lse[hrow] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <bool kNVFP4>
void launch_dim(const Plan& p, uint32_t grid, hipStream_t s) {
  switch (p.a.c.dim) {
    case 32: paged_decode_kernel<kNVFP4, 32><<<grid, kThreads, 0, s>>>(p); break;
    case 64: paged_decode_kernel<kNVFP4, 64><<<grid, kThreads, 0, s>>>(p); break;
    case 96: paged_decode_kernel<kNVFP4, 96><<<grid, kThreads, 0, s>>>(p); break;
    case 128: paged_decode_kernel<kNVFP4, 128><<<grid, kThreads, 0, s>>>(p); break;
    case 160: paged_decode_kernel<kNVFP4, 160><<<grid, kThreads, 0, s>>>(p); break;
    case 192: paged_decode_kernel<kNVFP4, 192><<<grid, kThreads, 0, s>>>(p); break;
    case 224: paged_decode_kernel<kNVFP4, 224><<<grid, kThreads, 0, s>>>(p); break;
    default: paged_decode_kernel<kNVFP4, 256><<<grid, kThreads, 0, s>>>(p); break;
  }
}

}  // namespace

int64_t decode_items(int64_t B, int64_t Hq, int64_t heads) {
  const int64_t G = Hq / heads;
  return kTargetItems + B * heads * ((G + kHeads - 1) / kHeads);
}

size_t decode_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t dim) {
  const int64_t G = Hq / heads;
  return sizeof(float) * (size_t)(decode_items(B, Hq, heads) * (G < kHeads ? G : kHeads) * (dim + 2));
}

hipError_t launch_paged_decode(const DecodeArgs& a, hipStream_t s) {
  Plan p;
  p.a = a;
  p.groups = (a.G + kHeads - 1) / kHeads;
  p.rows = a.G < kHeads ? a.G : kHeads;
  const uint64_t d = a.c.page_size / 8;
  p.page_magic = (((uint64_t)1 << 36) + d - 1) / d;
  // chunks: at most kTargetItems and one more for every sequence and head group, and
  // no more than the table's tokens give
  const int64_t cap = (int64_t)a.pages_per_seq * a.c.page_size;
  const int64_t heads = (int64_t)a.B * a.c.heads * p.groups;
  const int64_t most = (cap + kMinChunk - 1) / kMinChunk;
  const int64_t items = min(kTargetItems + heads, heads * max(most, (int64_t)1));
  if (a.c.nvfp4) launch_dim<true>(p, (uint32_t)items, s);
  else launch_dim<false>(p, (uint32_t)items, s);
  if (most > 1) join_kernel<<<(uint32_t)((int64_t)a.B * a.Hq), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace fos
