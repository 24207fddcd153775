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
constexpr int kChunkStep = 64 * kWaves;   // a step of every wave
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

// Tokens per chunk, a multiple of kChunkStep: enough that the batch gives about kTargetItems.
__device__ __forceinline__ int chunk_tokens(const Plan& p, int lane) {
  int64_t total = 0;
  for (int b = lane; b < p.a.B; b += 64) {
    const Range r = range_of(p, p.a.lens[b]);
    total += r.last - r.base;
  }
  total = wave_sum(total) * (p.a.c.heads * p.groups);
  int64_t c = (total + kTargetItems - 1) / kTargetItems;
  c = max(c, (int64_t)kMinChunk);
  c = (c + kChunkStep - 1) / kChunkStep * kChunkStep;
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

// E2M1 x E4M3 has at most 6 significant bits between 2^-10 and 2688: exact in half
// precision.
// Eight nibbles times the block scale in both halves of s.
__device__ __forceinline__ u32x4 dequant8(uint32_t w, f16x2 s) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
               __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}
// Byte kSel of w (two nibbles) times the two scales of s.
template <int kSel>
__device__ __forceinline__ uint32_t dequant2(uint32_t w, f16x2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, kSel) * s);
}
// The nibbles selected by 0x0f0f0f0f from x, the others from y.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t x, uint32_t y) {
  return (x & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
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

// Page id of the group of 8 tokens that starts at `tok` (a group never crosses a page)
// and the group's first row in the page; id -1 past `end`.
struct Group {
  int id, off;
};
__device__ __forceinline__ Group find_group(const Plan& p, const int32_t* table, int tok, int end) {
  const uint32_t g = (uint32_t)tok >> 3;
  const int page = (int)((g * p.page_magic) >> 36);
  Group x;
  x.id = tok < end ? table[page] : -1;
  x.off = tok - page * p.a.c.page_size;
  return x;
}
__device__ __forceinline__ bool held(const Plan& p, const Group& x) {
  return (uint32_t)x.id < (uint32_t)p.a.c.num_pages;   // num_pages < 2^31
}
// The group's first row in the cache; row 0 for a page that is not held (what is read
// there is masked).
__device__ __forceinline__ int64_t row_of(const Plan& p, const Group& x, int head) {
  return held(p, x) ? ((int64_t)x.id * p.a.c.heads + head) * p.a.c.page_size + x.off : 0;
}

// K and V of 32 tokens as one lane loads them: K rows as A operand rows, V rows of the
// lane's 8 tokens.
template <bool kNVFP4, int D>
struct Raw;
template <int D>
struct Raw<false, D> {
  using P = Pieces<D>;
  u32x4 k[2][D / 32];
  uint32_t v[8][D / 32];
  __device__ __forceinline__ void load_k(const KVCacheArgs& c, int64_t row, int q) {
    const uint16_t* base = reinterpret_cast<const uint16_t*>(c.k) + row * D + 8 * q;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        k[u][j] = *reinterpret_cast<const u32x4*>(base + 4 * u * D + 32 * j);
  }
  __device__ __forceinline__ void load_v(const KVCacheArgs& c, int64_t row, int r) {
    const uint16_t* base = reinterpret_cast<const uint16_t*>(c.v) + row * D;
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int n = P::size(i) / 16, at = P::at(i) / 32;   // values of the lane; its dwords
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t* w = base + P::at(i) + n * r + e * D;
        if (n == 8) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(w);
          v[e][at] = x.x; v[e][at + 1] = x.y; v[e][at + 2] = x.z; v[e][at + 3] = x.w;
        } else if (n == 4) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(w);
          v[e][at] = x.x; v[e][at + 1] = x.y;
        } else {
          v[e][at] = *reinterpret_cast<const uint32_t*>(w);
        }
      }
    }
  }
  __device__ __forceinline__ u32x4 k_step(int u, int j) const { return k[u][j]; }
  __device__ __forceinline__ void mask_v(uint32_t seen) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[e][i] = (seen >> e) & 1 ? v[e][i] : 0u;
  }
  // Tiles 2 i and 2 i + 1 of V^T: two values of each of the 8 tokens.
  __device__ __forceinline__ void v_tiles(int i, u32x4& even, u32x4& odd) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      even[e] = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x05040100u);
      odd[e] = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x07060302u);
    }
  }
};
template <int D>
struct Raw<true, D> {
  using P = Pieces<D>;
  uint32_t k[2][D / 32];           // 8 nibbles of each step
  uint32_t ks[2][P::count];        // one or two block scales of each piece
  uint32_t v[8][P::count];         // 8, 4 or 2 nibbles
  uint32_t vs[8][P::count];        // their block scale
  __device__ __forceinline__ void load_k(const KVCacheArgs& c, int64_t row, int q) {
    const uint8_t* base = c.k + row * (D / 2);
    const uint8_t* sbase = c.ks + row * (D / 16);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < P::count; ++i) {
        const int n = P::size(i) / 32, at = P::at(i) / 32;
        const uint8_t* w = base + 4 * u * (D / 2) + P::at(i) / 2 + 4 * n * q;
        const uint8_t* sp = sbase + 4 * u * (D / 16) + P::at(i) / 16;
        if (n == 4) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(w);
          k[u][at] = x.x; k[u][at + 1] = x.y; k[u][at + 2] = x.z; k[u][at + 3] = x.w;
          ks[u][i] = *reinterpret_cast<const uint16_t*>(sp + 2 * q);
        } else if (n == 2) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(w);
          k[u][at] = x.x; k[u][at + 1] = x.y;
          ks[u][i] = sp[q];
        } else {
          k[u][at] = *reinterpret_cast<const uint32_t*>(w);
          ks[u][i] = sp[q / 2];
        }
      }
  }
  __device__ __forceinline__ void load_v(const KVCacheArgs& c, int64_t row, int r) {
    const uint8_t* base = c.v + row * (D / 2);
    const uint8_t* sbase = c.vs + row * (D / 16);
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int n = P::size(i) / 16;
      const uint8_t* w = base + P::at(i) / 2 + n * r / 2;
      const uint8_t* sp = sbase + (P::at(i) + n * r) / 16;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint8_t* we = w + e * (D / 2);
        v[e][i] = n == 8 ? *reinterpret_cast<const uint32_t*>(we)
                  : n == 4 ? *reinterpret_cast<const uint16_t*>(we) : *we;
        vs[e][i] = sp[e * (D / 16)];
      }
    }
  }
  __device__ __forceinline__ u32x4 k_step(int u, int j) const {
    int i = 0;
#pragma unroll
    for (int x = 1; x < P::count; ++x) i = 32 * j >= P::at(x) ? x : i;
    const int in = j - P::at(i) / 32;          // step of the piece
    const f16x2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(ks[u][i], 1.0f, false);
    const _Float16 x = in >= 2 ? s.y : s.x;
    return dequant8(k[u][j], f16x2{x, x});
  }
  __device__ __forceinline__ void mask_v(uint32_t seen) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < P::count; ++i) vs[e][i] = (seen >> e) & 1 ? vs[e][i] : 0u;
  }
  // The nibbles of two tokens are brought together (four tokens' worth of bit selects for
  // eight conversions), so that one conversion gives two tokens of one d.
  __device__ __forceinline__ void v_tiles(int t, u32x4& even, u32x4& odd) const {
    int i = 0;
#pragma unroll
    for (int x = 1; x < P::count; ++x) i = 32 * t >= P::at(x) ? x : i;
    const int sel = t - P::at(i) / 32;         // byte of the word
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f16x2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(vs[2 * e][i] | vs[2 * e + 1][i] << 8,
                                                               1.0f, false);
      const uint32_t a = low_nibbles(v[2 * e][i], v[2 * e + 1][i] << 4);
      const uint32_t b = low_nibbles(v[2 * e][i] >> 4, v[2 * e + 1][i]);
      even[e] = sel == 0 ? dequant2<0>(a, s) : sel == 1 ? dequant2<1>(a, s)
                : sel == 2 ? dequant2<2>(a, s) : dequant2<3>(a, s);
      odd[e] = sel == 0 ? dequant2<0>(b, s) : sel == 1 ? dequant2<1>(b, s)
               : sel == 2 ? dequant2<2>(b, s) : dequant2<3>(b, s);
    }
  }
};

// Tokens of one step of a wave: 64 of an NVFP4 cache of up to 128 values, else 32 (the
// K and V of a step are held in registers).
template <bool kNVFP4, int D>
constexpr int kSub = kNVFP4 && D <= 128 ? 2 : 1;
// Waves per SIMD that the registers are shared out for.
template <bool kNVFP4, int D>
constexpr int kMinWaves = !kNVFP4 && D > 160 ? 1 : 2;
constexpr float kSlack = 8.0f;    // see the rescaling below

template <bool kNVFP4, int D>
__global__ __launch_bounds__(kThreads, (kMinWaves<kNVFP4, D>)) void paged_decode_kernel(Plan p) {
  constexpr int kSteps = D / 32;               // 32-value steps of the first product
  constexpr int kTiles = D / 16;               // 16-row tiles of the second
  constexpr int kPad = D + 4;
  constexpr int N = kSub<kNVFP4, D>;
  using P = Pieces<D>;
  __shared__ __attribute__((aligned(16))) float so[kWaves][kHeads][kPad];
  __shared__ float sm[kWaves][kHeads], sl[kWaves][kHeads];
  const DecodeArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int chunk = chunk_tokens(p, lane);
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

  // Pipeline of a wave's steps: page ids two steps ahead, K one step ahead from the end of
  // the first product, V from the end of the second.
  constexpr int kStride = 32 * N * kWaves;
  Raw<kNVFP4, D> raw[N];
  Group gk[N], gv[N];
  bool v_held[N];
  auto find = [&](int t) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      gk[n] = find_group(p, table, t + 32 * n + 8 * (r >> 2), end);
      gv[n] = find_group(p, table, t + 32 * n + 8 * q, end);
    }
  };
  auto load_k = [&]() {
#pragma unroll
    for (int n = 0; n < N; ++n) raw[n].load_k(a.c, row_of(p, gk[n], head) + (r & 3), q);
  };
  auto load_v = [&](const Group (&g)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) raw[n].load_v(a.c, row_of(p, g[n], head), r);
  };
  int t = begin + 32 * N * wave;
  if (t < end) {
    find(t);
    load_k();
    load_v(gv);
#pragma unroll
    for (int n = 0; n < N; ++n) v_held[n] = held(p, gv[n]);
    find(t + kStride);
  }
  for (; t < end; t += kStride) {
    uint32_t seen[N];                          // bit e: token e of the lane is visible
    bool all = true;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int tok = t + 32 * n + 8 * q;      // visible: tokens first .. end - 1 of the 8
      const int lo = min(max(rg.first - tok, 0), 8), hi = min(max(end - tok, 0), 8);
      seen[n] = v_held[n] ? (0xffu >> (8 - hi)) & (0xffu << lo) & 0xffu : 0u;
      all = all && seen[n] == 0xffu;
    }
    all = __all(all);

    // scores in powers of two
    float w[N][8];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) s = mfma<kNVFP4>(raw[n].k_step(u, j), qf[j], s);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[n][4 * u + i] = s[i] * cs;
      }
    // the next step's page ids have arrived: its K, and the ids after it
    const bool more = t + kStride < end;       // the same for every lane
    Group next_v[N];
    if (more) {
      load_k();
#pragma unroll
      for (int n = 0; n < N; ++n) next_v[n] = gv[n];
      find(t + 2 * kStride);
    }
    if (!all) {
      asm volatile("");                        // a branch, not selects in every step
#pragma unroll
      for (int n = 0; n < N; ++n) {
        raw[n].mask_v(seen[n]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[n][e] = (seen[n] >> e) & 1 ? w[n][e] : -INFINITY;
      }
    }
    // Rescaling.  m is a common reference of a head's four lanes rather than the exact
    // maximum: it moves only when a score is more than 2^kSlack above it, so that most
    // steps need neither the exchange between the lanes nor the products with o.  Weights
    // are then at most 2^kSlack, well inside half precision.
    float top = w[0][0];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, w[n][e]);
    if (__any(top > m + kSlack)) {
      const float m2 = fmaxf(m, max_over_groups(top));
      const float f = m2 == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) o[i] *= f;
    }
    const float m0 = m == -INFINITY ? 0.0f : m;
    // weights of the second product: half precision (11 bits) beside exact half-precision
    // V; beside bf16 V as the sum of two bf16 (16 bits), since one would round the weights
    // to 8 bits
    u32x4 hi[N], lo[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[n][e] = __builtin_amdgcn_exp2f(w[n][e] - m0);
        l += w[n][e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = w[n][2 * e], y = w[n][2 * e + 1];
        if constexpr (kNVFP4) {
          hi[n][e] = pack_f16x2(x, y);
        } else {
          hi[n][e] = pack_bf16x2(x, y);
          lo[n][e] = pack_bf16x2(x - bf16_lo(hi[n][e]), y - bf16_hi(hi[n][e]));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        u32x4 even, odd;
        raw[n].v_tiles(i, even, odd);
        o[2 * i] = mfma<kNVFP4>(even, hi[n], o[2 * i]);
        o[2 * i + 1] = mfma<kNVFP4>(odd, hi[n], o[2 * i + 1]);
        if constexpr (!kNVFP4) {
          o[2 * i] = mfma<false>(even, lo[n], o[2 * i]);
          o[2 * i + 1] = mfma<false>(odd, lo[n], o[2 * i + 1]);
        }
      }
    if (more) {
      load_v(next_v);
#pragma unroll
      for (int n = 0; n < N; ++n) v_held[n] = held(p, next_v[n]);
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
  const int chunk = chunk_tokens(p, lane);
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
