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
// Split.  The steps (256 tokens) of all sequences form one list, and for every kv head
// the workgroups that the GPU holds at once take equal runs of it: all start together and
// all are done together, however ragged the lengths are.  Where runs that end with their
// sequence are hardly longer, these are taken.  The lengths are read on the device; the
// host needs none.  Workgroups of the same run and neighbouring heads are neighbours: they
// read the same pages at the same time.  A sequence that fell to several runs leaves partial
// (m, l, o) in the workspace, and the last workgroup to finish joins them (of many, in two
// levels) in their order: no second launch, nobody waits, and the order of every sum
// depends on the lengths and the call's sizes (heads, dim, batch, width of the table) alone.
//
// Bound and figures (K and V bytes over the time of a launch).  bf16: memory; 32 sequences
// of up to 8192 tokens, 32 heads over 8 of 128: 90 us, 6.0 TB/s of 6.8 that a plain read
// reaches.  NVFP4: the loads and the conversions of their step share the time; 16 x up to
// 32768 tokens, 64 heads over 8 of 128: 63 us, 4.9 TB/s (55 us with the arithmetic left
// out; VALU work in 62% of the cycles).  Few tokens (1 x 200): 6.5 us, of which an empty
// launch is 2.
#include <cfloat>

#include "serving.hpp"

namespace fos {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kHeads = 16;            // query heads per workgroup: columns of the products
constexpr int kStepTokens = 64 * kWaves;   // a step of a workgroup
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

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
  int runs;                // per head group
  uint32_t* arrived;       // per segment: workgroups done with it, 0 between launches
  uint32_t* grouped;       // the same for a group of partials (below)
  float* parts;
  float* group_parts;
};

// Partial results: o[rows][dim], (m, l)[rows], padded to 16 bytes.  Run i of a head group
// leaves the one of sequence b at i + b: along the list one of the two grows from each to
// the next, so the places are distinct, and those of a sequence lie in a row.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) {
  return (int64_t)rows * dim + ((2 * rows + 3) & ~3);
}
__device__ __forceinline__ int64_t part_stride(const Plan& p) {
  return part_floats(p.rows, p.a.c.dim);
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

// Inclusive sum over the lanes (DPP: within rows of 16, then from row to row).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast 15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast 31
  return v;
}
// Steps of a sequence of this length for one head, at most 2^22; an empty one takes a
// step to write its zeros.
__device__ __forceinline__ int steps_of(const Plan& p, int len) {
  const Range r = range_of(p, len);
  return max(1, (r.last - r.base + kStepTokens - 1) / kStepTokens);
}
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A workgroup's run [pos, end) of the list of steps, and its current sequence: steps
// [at, at + steps) of the list are sequence b, `len` tokens.  The API keeps the list below
// 2^31.  Every lane of a wave holds the same values, but for sum and upto: lane i's share
// of the sequences, i * each and on.
struct Run {
  int each, sum, upto, len0;
  int share, pos, end;
  int b, len, steps, at;
  bool one;                // the run is one piece of a sequence: at = 0, and these count it
  int first, count;        // run of the sequence's first piece, its pieces
};
// A run that spans two sequences pays for the start of a second pipeline and for a second
// result, about as much as two steps of an NVFP4 cache and less than one of a bf16 cache.
// Where runs of one piece each, at most this much longer, are enough for all sequences,
// these are taken (24 x 12 heads x the last 1000 tokens of 96 values, NVFP4: 20.1 -> 18.2
// us; 32 x 8 heads x 4000 of 64, bf16: 48.4 -> 46.9; a bf16 step longer than the equal
// share, 32 x 8 x up to 8192 of 128: 93.1 instead of 89.5).
template <bool kNVFP4>
constexpr int kRestart = kNVFP4 ? 2 : 0;
template <bool kNVFP4>
__device__ __forceinline__ void begin_run(const Plan& p, Run& u, int run) {
  const int lane = threadIdx.x & 63, B = p.a.B;
  u.each = (B + 63) >> 6;
  u.sum = u.len0 = 0;
  for (int i = 0; i < u.each; ++i) {
    const int b = lane * u.each + i;
    if (b < B) {
      u.len0 = p.a.lens[b];
      u.sum += steps_of(p, u.len0);
    }
  }
  u.upto = wave_scan(u.sum);
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane(u.upto, 63);
  u.share = scalar((int)((total + p.runs - 1) / (uint32_t)p.runs));
  u.one = false;
  if (u.each == 1 && u.share > 1) {
    for (int more = 0; more <= kRestart<kNVFP4>; ++more) {
      const int share = u.share + more;
      const int n = (int)((uint32_t)(u.sum + share - 1) / (uint32_t)share), upto = wave_scan(n);
      if (__builtin_amdgcn_readlane(upto, 63) > p.runs) continue;
      u.one = true;
      u.pos = u.end = u.at = 0;
      const uint64_t hit = __ballot(run >= upto - n && run < upto);
      if (hit == 0) return;
      u.b = __ffsll((unsigned long long)hit) - 1;
      u.len = __builtin_amdgcn_readlane(u.len0, u.b);
      u.steps = __builtin_amdgcn_readlane(u.sum, u.b);
      u.count = __builtin_amdgcn_readlane(n, u.b);
      u.first = __builtin_amdgcn_readlane(upto, u.b) - u.count;
      u.pos = (run - u.first) * share;
      u.end = min(u.pos + share, u.steps);
      return;
    }
  }
  // unsigned: runs * share is below 2^31 + runs
  const uint32_t pos = (uint32_t)run * (uint32_t)u.share;
  u.pos = (int)min(pos, total);
  u.end = (int)min(pos + (uint32_t)u.share, total);
}
// The sequence at u.pos.
__device__ __forceinline__ void find_sequence(const Plan& p, Run& u) {
  const int lane = threadIdx.x & 63, y = u.pos;
  int start = u.upto - u.sum;
  const int l = __ffsll((unsigned long long)__ballot(y >= start && y < u.upto)) - 1;
  start = __builtin_amdgcn_readlane(start, l);
  if (u.each == 1) {
    u.b = l;
    u.len = __builtin_amdgcn_readlane(u.len0, l);
    u.steps = __builtin_amdgcn_readlane(u.sum, l);
  } else {
    for (int i = 0; i < u.each; i += 64) {
      const int b = l * u.each + i + lane;
      const bool in = i + lane < u.each && b < p.a.B;
      const int len = in ? p.a.lens[b] : 0, n = in ? steps_of(p, len) : 0;
      const int upto = start + wave_scan(n);
      const uint64_t hit = __ballot(y >= upto - n && y < upto);
      if (hit) {
        const int k = __ffsll((unsigned long long)hit) - 1;
        u.b = l * u.each + i + k;
        u.len = __builtin_amdgcn_readlane(len, k);
        u.steps = __builtin_amdgcn_readlane(n, k);
        start = __builtin_amdgcn_readlane(upto - n, k);
        break;
      }
      start = __builtin_amdgcn_readlane(upto, 63);
    }
  }
  u.at = start;
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
// The same as bf16, where it is exact too.
__device__ __forceinline__ u32x4 dequant8_bf16(uint32_t w, float s) {
  const f32x2 a = cvt_pk_f32_fp4<0>(w), b = cvt_pk_f32_fp4<1>(w);
  const f32x2 c = cvt_pk_f32_fp4<2>(w), d = cvt_pk_f32_fp4<3>(w);
  return u32x4{pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s),
               pack_bf16x2(c.x * s, c.y * s), pack_bf16x2(d.x * s, d.y * s)};
}
constexpr int kShiftBf16 = 12;    // 6 * 448 < 2^12
// Byte kSel of w (two nibbles) times the two scales of s.
template <int kSel>
__device__ __forceinline__ uint32_t dequant2(uint32_t w, f16x2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, kSel) * s);
}
// The two E4M3 scales in the low or high half of w.
__device__ __forceinline__ f16x2 scale_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}
__device__ __forceinline__ f16x2 scale_pair_hi(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
}
// The nibbles selected by 0x0f0f0f0f from x, the others from y.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t x, uint32_t y) {
  return (x & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
}

// The smaller of m and the magnitudes of two bf16 less 1 (a zero: the largest), by halves.
__device__ __forceinline__ uint32_t pk_min_less1(uint32_t m, uint32_t w) {
  const u16x2 b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu) - u16x2{1, 1};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, m), b));
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

// K and V of one step of a wave (kTokens tokens), on their way from memory to the
// operands.  A load instruction whose neighbouring lanes sit in different rows costs the
// address unit a line per lane, so what an operand wants row by row (K, and everything of
// an NVFP4 cache: its rows are short) is loaded in memory order, 16 bytes per lane, and
// goes through the wave's own piece of LDS.  Loads stay in registers until the next step,
// and are non-temporal: K and V are read once (5.9 -> 6.8 TB/s for a plain read of 300 MB).
//
// 16-byte units of a row are stored at (unit ^ key): with the key of the row below, the 16
// rows of an operand read start in different banks.
__host__ __device__ constexpr int pow2_part(int n) { return n & -n; }

template <bool kNVFP4, int D>
struct Step;

template <int D>
struct Step<false, D> {
  using P = Pieces<D>;
  static constexpr int kTokens = 32;
  static constexpr int kUnits = D / 8;               // 16-byte units of a K row
  static constexpr int kLoads = D / 16;              // units of a lane: 32 * kUnits / 64
  static constexpr int kLds = kTokens * D * 2;       // K
  u32x4 kr[kLoads];
  uint32_t v[8][D / 32];                             // V: rows of the lane's 8 tokens
  static __device__ __forceinline__ int key(int row) {
    return ((row >> 3) << 2 | (row & 3)) & (pow2_part(kUnits) - 1);
  }
  __device__ __forceinline__ void load(const KVCacheArgs& c, uint32_t row8, int lane) {
    const u32x4* kb = reinterpret_cast<const u32x4*>(c.k);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = lane + 64 * i, row = at / kUnits, u = at % kUnits;
      const uint32_t r8 = __shfl(row8, row >> 3);
      kr[i] = __builtin_nontemporal_load(kb + ((uint64_t)r8 * 8 + (row & 7)) * kUnits + u);
    }
  }
  // V of the next step, once this one's is used
  __device__ __forceinline__ void load_late(const KVCacheArgs& c, uint32_t row8, int lane) {
    const int r = lane & 15, q = lane >> 4;
    const uint16_t* vb =
        reinterpret_cast<const uint16_t*>(c.v) + (uint64_t)__shfl(row8, q) * (8 * D);
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int n = P::size(i) / 16, at = P::at(i) / 32;   // values of the lane; its dwords
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t* w = vb + P::at(i) + n * r + e * D;
        if (n == 8) {
          const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w));
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
  __device__ __forceinline__ void stage(uint8_t* lds, int lane) {
    u32x4* l = reinterpret_cast<u32x4*>(lds);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = lane + 64 * i, row = at / kUnits, u = at % kUnits;
      l[row * kUnits + (u ^ key(row))] = kr[i];
    }
  }
  // Scores of 16 tokens: operand rows r = tokens 8 (r / 4) + 4 u + r % 4.
  __device__ __forceinline__ f32x4 scores(const uint8_t* lds, const u32x4 (&qf)[D / 32], int,
                                          int u, int r, int q) const {
    const int row = 8 * (r >> 2) + 4 * u + (r & 3);
    const u32x4* l = reinterpret_cast<const u32x4*>(lds) + row * kUnits;
    f32x4 s = {0, 0, 0, 0};
    u32x4 k[D / 32];                           // all on their way before the first product
#pragma unroll
    for (int j = 0; j < D / 32; ++j) k[j] = l[(4 * j + q) ^ key(row)];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) s = mfma<false>(k[j], qf[j], s);
    return s;
  }
  __device__ __forceinline__ void mask_v(uint8_t*, const uint32_t* seen, int) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[e][i] = (seen[0] >> e) & 1 ? v[e][i] : 0u;
  }
  // o += V^T P^T: tiles 2 i and 2 i + 1 take two values of each of the 8 tokens.
  __device__ __forceinline__ void accumulate(const uint8_t*, f32x4 (&o)[D / 16], int,
                                             const u32x4& hi, const u32x4& lo, int, int) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      u32x4 even, odd;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        even[e] = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x05040100u);
        odd[e] = __builtin_amdgcn_perm(v[2 * e + 1][i], v[2 * e][i], 0x07060302u);
      }
      o[2 * i] = mfma<false>(even, hi, o[2 * i]);
      o[2 * i + 1] = mfma<false>(odd, hi, o[2 * i + 1]);
      o[2 * i] = mfma<false>(even, lo, o[2 * i]);
      o[2 * i + 1] = mfma<false>(odd, lo, o[2 * i + 1]);
    }
  }
};

template <int D>
struct Step<true, D> {
  using P = Pieces<D>;
  static constexpr int kTokens = 64, N = kTokens / 32;
  static constexpr int kRow = D / 2;                 // bytes of a row
  static constexpr int kUnits = D / 32;              // its 16-byte units, and those of a lane
  static constexpr int kBlocks = D / 16;             // its block scales
  // LDS: K, V, their scales as in memory, V's scales by block
  static constexpr int kV = kTokens * kRow, kKS = 2 * kV, kVR = kKS + kTokens * kBlocks;
  static constexpr int kVS = kVR + kTokens * kBlocks;
  static constexpr int kLds = kVS + kTokens * kBlocks;
  u32x4 kr[kUnits], vr[kUnits];
  // Block scales: 8 rows are kUnits units (rows alone may start at any even byte, and loads
  // off their alignment take several times as long: 18 us with aligned loads against 33
  // with 6-byte ones, 24 x 12 heads x 1000 tokens of 96 values).  K's and V's in one load
  // where both have the lanes.
  static constexpr int kScaleUnits = 8 * kUnits;     // of K, and of V
  static constexpr bool kOneLoad = 2 * kScaleUnits <= 64;
  u32x4 sr[kOneLoad ? 1 : 2];
  static __device__ __forceinline__ int key(int row) { return (row >> 3) & 3 & (pow2_part(kUnits) - 1); }
  __device__ __forceinline__ void load(const KVCacheArgs& c, uint32_t row8, int lane) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int at = lane + 64 * i, row = at / kUnits, u = at % kUnits;
      const uint64_t g = ((uint64_t)__shfl(row8, row >> 3) * 8 + (row & 7)) * kUnits + u;
      kr[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.k) + g);
      vr[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.v) + g);
    }
    const int at = kOneLoad ? lane % kScaleUnits : lane;
    const uint64_t g = (uint64_t)__shfl(row8, at / kUnits) * kUnits + at % kUnits;
    if constexpr (kOneLoad) {
      if (lane < 2 * kScaleUnits)
        sr[0] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(lane < kScaleUnits ? c.ks : c.vs) + g);
    } else if (lane < kScaleUnits) {
      sr[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.ks) + g);
      sr[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.vs) + g);
    }
  }
  __device__ __forceinline__ void load_late(const KVCacheArgs&, uint32_t, int) {}
  // K scales as they are ([token][block]); V scales by block ([block][token]), so that a
  // lane reads the scales of its 8 tokens at once.
  __device__ __forceinline__ void stage(uint8_t* lds, int lane) {
    u32x4* l = reinterpret_cast<u32x4*>(lds);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int at = lane + 64 * i, row = at / kUnits, u = at % kUnits;
      l[row * kUnits + (u ^ key(row))] = kr[i];
      l[kV / 16 + row * kUnits + (u ^ key(row))] = vr[i];
    }
    if constexpr (kOneLoad) {
      if (lane < 2 * kScaleUnits) l[kKS / 16 + lane] = sr[0];
    } else if (lane < kScaleUnits) {
      l[kKS / 16 + lane] = sr[0];
      l[kKS / 16 + kScaleUnits + lane] = sr[1];
    }
    // transpose V's: a lane takes a token
    const uint16_t* sp = reinterpret_cast<const uint16_t*>(lds + kVR + lane * kBlocks);
    uint16_t row[kBlocks / 2];
    __builtin_memcpy(row, __builtin_assume_aligned(sp, pow2_part(kBlocks)), kBlocks);
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      lds[kVS + i * kTokens + lane] = (uint8_t)(row[i / 2] >> (8 * (i % 2)));
  }
  // The operands of a step as they lie in LDS.  They are all read before the first product:
  // left where they are used, every read is waited for, and with one or two waves on a SIMD
  // little else runs meanwhile (24 x 12 heads x 1000 tokens of 96 values: 18.2 -> 17.0 us,
  // 16 x 8 heads x 32768 of 128: 64.0 -> 61.7).
  uint32_t kw[2 * N][D / 32], vw[N][P::count][8];
  uint16_t ksc[2 * N][P::count];
  u32x2 vsc[N][P::count];
  // K of 16 tokens: operand rows r = tokens 8 (r / 4) + 4 u + r % 4 of the 32.
  __device__ __forceinline__ void read_k(const uint8_t* lds, int n, int u, int r, int q) {
    const int row = 32 * n + 8 * (r >> 2) + 4 * u + (r & 3), t = 2 * n + u;
    const uint8_t* l = lds + row * kRow;
    const uint8_t* sp = lds + kKS + row * kBlocks;
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int steps = P::size(i) / 32, j0 = P::at(i) / 32;
      // the lane's 4 * steps bytes of the piece: in unit j0 + steps q / 4
      const uint8_t* w = l + 16 * ((j0 + steps * q / 4) ^ key(row)) + (4 * steps * q) % 16;
      if (steps == 4) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(w);
        kw[t][j0] = x.x; kw[t][j0 + 1] = x.y; kw[t][j0 + 2] = x.z; kw[t][j0 + 3] = x.w;
        ksc[t][i] = *reinterpret_cast<const uint16_t*>(sp + 2 * j0 + 2 * q);
      } else if (steps == 2) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(w);
        kw[t][j0] = x.x; kw[t][j0 + 1] = x.y;
        ksc[t][i] = sp[2 * j0 + q];
      } else {
        kw[t][j0] = *reinterpret_cast<const uint32_t*>(w);
        ksc[t][i] = sp[2 * j0 + q / 2];
      }
    }
  }
  // V of the lane's 8 tokens of the 32.
  __device__ __forceinline__ void read_v(const uint8_t* lds, int n, int r, int q) {
    const int tok = 32 * n + 8 * q;                  // one key for the group's 8 rows
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int bytes = P::size(i) / 32;             // of the lane and token: 4, 2 or 1
      const int b = P::at(i) / 2 + bytes * r;
      const uint8_t* w = lds + kV + tok * kRow + 16 * ((b / 16) ^ key(tok)) + b % 16;
      vsc[n][i] = *reinterpret_cast<const u32x2*>(lds + kVS + (b / 8) * kTokens + tok);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (bytes == 4) vw[n][i][e] = *reinterpret_cast<const uint32_t*>(w + e * kRow);
        else if (bytes == 2) vw[n][i][e] = *reinterpret_cast<const uint16_t*>(w + e * kRow);
        else vw[n][i][e] = w[e * kRow];
      }
    }
  }
  __device__ __forceinline__ void read_all(const uint8_t* lds, int r, int q) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) read_k(lds, n, u, r, q);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < N; ++n) read_v(lds, n, r, q);
  }
  __device__ __forceinline__ f32x4 scores(const uint8_t*, const u32x4 (&qf)[D / 32], int n, int u,
                                          int, int) const {
    f32x4 s = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const f16x2 sc = scale_pair(ksc[2 * n + u][i]);
#pragma unroll
      for (int j = 0; j < P::size(i) / 32; ++j) {
        const _Float16 x = j >= 2 ? sc.y : sc.x;
        const int at = P::at(i) / 32 + j;
        s = mfma<true>(dequant8(kw[2 * n + u][at], f16x2{x, x}), qf[at], s);
      }
    }
    return s;
  }
  // The same for queries that half precision cannot hold: bf16 operands.  K is exact in
  // them too, but its block scale is applied in fp32, value by value.  K enters times
  // 2^-kShiftBf16, below 1, so that a product with any query is finite.
  __device__ __forceinline__ f32x4 scores_bf16(const u32x4 (&qf)[D / 32], int n, int u) const {
    f32x4 s = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const f32x2 sc = __builtin_amdgcn_cvt_pk_f32_fp8(ksc[2 * n + u][i], false) *
                       __builtin_ldexpf(1.0f, -kShiftBf16);
#pragma unroll
      for (int j = 0; j < P::size(i) / 32; ++j) {
        const int at = P::at(i) / 32 + j;
        s = mfma<false>(dequant8_bf16(kw[2 * n + u][at], j >= 2 ? sc.y : sc.x), qf[at], s);
      }
    }
    return s;
  }
  __device__ __forceinline__ void mask_v(uint8_t* lds, const uint32_t* seen, int lane) {
    // lane r < 8 of group q holds the mask of groups q and 4 + q of 8 tokens: each of the
    // group's 16 lanes clears the scales of one token and half
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int tok = 32 * n + 8 * (lane >> 4) + (lane & 7);
      if ((lane & 8) == 0 && !((seen[n] >> (lane & 7)) & 1)) {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) lds[kVS + i * kTokens + tok] = 0;
      }
    }
  }
  // The nibbles of two tokens are brought together (four bit selects for eight
  // conversions), so that one conversion gives two tokens of one d.
  __device__ __forceinline__ void accumulate(const uint8_t*, f32x4 (&o)[D / 16], int n,
                                             const u32x4& hi, const u32x4&, int, int) const {
#pragma unroll
    for (int i = 0; i < P::count; ++i) {
      const int bytes = P::size(i) / 32;             // of the lane and token: 4, 2 or 1
      const u32x2 sb = vsc[n][i];
      uint32_t lo[4], up[4];
      f16x2 sc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = vw[n][i][2 * e], y = vw[n][i][2 * e + 1];
        lo[e] = low_nibbles(x, y << 4);
        up[e] = low_nibbles(x >> 4, y);
        sc[e] = e & 1 ? scale_pair_hi(sb[e / 2]) : scale_pair(sb[e / 2]);
      }
#pragma unroll
      for (int j = 0; j < bytes; ++j) {
        u32x4 even, odd;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          even[e] = j == 0 ? dequant2<0>(lo[e], sc[e]) : j == 1 ? dequant2<1>(lo[e], sc[e])
                    : j == 2 ? dequant2<2>(lo[e], sc[e]) : dequant2<3>(lo[e], sc[e]);
          odd[e] = j == 0 ? dequant2<0>(up[e], sc[e]) : j == 1 ? dequant2<1>(up[e], sc[e])
                   : j == 2 ? dequant2<2>(up[e], sc[e]) : dequant2<3>(up[e], sc[e]);
        }
        const int t = P::at(i) / 16 + 2 * j;
        o[t] = mfma<true>(even, hi, o[t]);
        o[t + 1] = mfma<true>(odd, hi, o[t + 1]);
      }
    }
  }
};

constexpr float kSlack = 8.0f, kBelow = 7.0f;    // see the rescaling below

// Joining partials.  A thread takes four values of a head and reads kBatch partials at a
// time; where that leaves threads idle, `split` of them share the partials of the same
// values.  A segment of many partials is joined in two levels, by the last workgroup of
// each group of `size` partials and by the last of the groups: what counts is how many
// rounds of reads follow one another (1 x 41461 tokens, bf16, 2 kv heads of 192 values with
// 16 query heads each: 50 us on one level, 30 on two; 2 x up to 27428, NVFP4, 1 head of 256:
// 18.5 and 14.3, and 22.7 if threads do not share).  More partials at a time cost more where
// there are two or three than they save elsewhere (24 x 12 heads x 1000 x 64: 12.8 us with
// 4, 13.1 with 8).
constexpr int kBatch = 4;
struct Joining {
  int split, size, groups;
};
template <int D>
__device__ __forceinline__ Joining plan_joining(int rows, int count) {
  const int items = rows * (D / 4);
  Joining j;
  const int most = items <= 32 ? 8 : items <= 64 ? 4 : items <= 128 ? 2 : 1;
  j.split = 1;
  while (j.split < most && kBatch * j.split < count) j.split *= 2;
  const int unit = kBatch * j.split, passes = (items + kThreads - 1) / kThreads;
  j.size = count;
  j.groups = 1;
  if (count > 2 * unit) {
    int size = unit;
    while (2 * size * size < count) size *= 2;
    const int groups = (int)((uint32_t)(count + size - 1) / (uint32_t)size);
    const int one = (count + unit - 1) / unit;
    const int two = (size + unit - 1) / unit + (groups + unit - 1) / unit;
    if (passes * one > passes * two + 1) {
      j.size = size;
      j.groups = groups;
    }
  }
  return j;
}

struct Joined {
  float m, l;
  f32x4 o;
};
// The sum of a and b with the common maximum.
__device__ __forceinline__ void add(Joined& a, const Joined& b) {
  const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.0f : m;
  const float fa = __builtin_amdgcn_exp2f(a.m - ref), fb = __builtin_amdgcn_exp2f(b.m - ref);
  a.l = a.l * fa + b.l * fb;
  a.o = a.o * fa + b.o * fb;
  a.m = m;
}

// Joins `count` partials, in an order that depends on their number alone: into a partial
// at `to`, or (null) into the outputs.  Called by the whole workgroup.
template <int D>
__device__ __forceinline__ void join_partials(const Plan& p, const float* all, int count, int split,
                                              int rows, float* to, int64_t hrow0, float vt0,
                                              Joined* scratch) {
  const int step = 4 * (int)part_stride(p);      // bytes; all of a segment are below 2^24
  const __amdgpu_buffer_rsrc_t parts = shared_floats(all, count * step);
  const int items = rows * (D / 4);
  int tid = threadIdx.x;
  asm("" : "+v"(tid));       // what depends on it is not to be kept through the steps
  // partials sub, sub + split, .. of item i
  auto gather = [&](int i, int sub) {
    const int g = i / (D / 4), d = 4 * (i % (D / 4));
    Joined r{-INFINITY, 0.0f, {0, 0, 0, 0}};
    for (int c = sub; c < count; c += kBatch * split) {
      f32x2 ml[kBatch];
      f32x4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int at = min(c + k * split, count - 1) * step;
        ml[k] = load_shared2(parts, at + 4 * (p.rows * D + 2 * g));
        x[k] = load_shared4(parts, at + 4 * (g * D + d));
      }
      float m = r.m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) m = fmaxf(m, ml[k].x);
      const float ref = m == -INFINITY ? 0.0f : m;       // nothing seen so far: all weights 0
      const float f = __builtin_amdgcn_exp2f(r.m - ref);
      r.m = m;
      r.l *= f;
      r.o *= f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = c + k * split < count ? __builtin_amdgcn_exp2f(ml[k].x - ref) : 0.0f;
        r.l += w * ml[k].y;
        r.o += w * x[k];
      }
    }
    return r;
  };
  auto finish = [&](int i, const Joined& r) {
    const int g = i / (D / 4), d = 4 * (i % (D / 4));
    if (to) {
      store_shared(to + g * D + d, f32x2{r.o[0], r.o[1]});
      store_shared(to + g * D + d + 2, f32x2{r.o[2], r.o[3]});
      if (d == 0) store_shared(to + p.rows * D + 2 * g, f32x2{r.m, r.l});
      return;
    }
    const float n = r.l == 0.0f ? 0.0f : vt0 / r.l;      // a NaN sum stays one
    *reinterpret_cast<u32x2*>(p.a.out + (hrow0 + g) * D + d) =
        u32x2{pack_bf16x2(r.o[0] * n, r.o[1] * n), pack_bf16x2(r.o[2] * n, r.o[3] * n)};
    if (d == 0 && p.a.lse)
      p.a.lse[hrow0 + g] = r.l == 0.0f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
  };
  if (split == 1) {
    for (int i = tid; i < items; i += kThreads) finish(i, gather(i, 0));
  } else {
    const int sub = tid / items;
    if (sub < split) scratch[tid] = gather(tid - sub * items, sub);
    __syncthreads();
    if (tid < items) {
      Joined r = scratch[tid];
      for (int s = 1; s < split; ++s) add(r, scratch[tid + s * items]);
      finish(tid, r);
    }
  }
}

// Workgroups that a CU holds at once: what the registers of a step leave room for (two
// with spills, NVFP4: 20.9 us instead of 18.4 at 8 x 4 heads x 8000 x 160, 34.4 instead of
// 20.6 at 192).
template <int D>
constexpr int kPerCU = D <= 64 ? 3 : D <= 128 ? 2 : 1;

template <bool kNVFP4, int D>
__global__ __launch_bounds__(kThreads, kPerCU<D>) void paged_decode_kernel(Plan p) {
  constexpr int kSteps = D / 32;               // 32-value steps of the first product
  constexpr int kTiles = D / 16;               // 16-row tiles of the second
  constexpr int kPad = D + 4;
  using P = Pieces<D>;
  using S = Step<kNVFP4, D>;
  constexpr int N = S::kTokens / 32;
  constexpr int kJoin = kHeads * kPad * 4;     // bytes of a wave's o
  // the waves' pieces during the steps, their o after them
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * (S::kLds > kJoin ? S::kLds : kJoin)];
  __shared__ float sm[kWaves][kHeads], sl[kWaves][kHeads];
  __shared__ uint32_t before_me;
  const DecodeArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const float kt0 = kNVFP4 ? a.c.kt[0] : 1.0f, vt0 = kNVFP4 ? a.c.vt[0] : 1.0f;
  const int per = a.c.heads * p.groups, hg = blockIdx.x % per;
  const int head = hg / p.groups, g0 = (hg % p.groups) * kHeads;
  const int rows = min(kHeads, a.G - g0);
  Run run;
  begin_run<kNVFP4>(p, run, blockIdx.x / per);
  for (; run.pos < run.end; __syncthreads()) {
  if (!run.one) find_sequence(p, run);
  const Range rg = range_of(p, run.len);
  // this workgroup's tokens of the sequence (at most 2^30, and a step more)
  const int steps = min(run.at + run.steps, run.end) - run.pos;
  const int begin = rg.base + (run.pos - run.at) * kStepTokens;
  const int end = min(rg.last, begin + steps * kStepTokens);
  const bool whole = steps == run.steps;
  const int32_t* table = a.table + run.b * a.table_stride;

  // Pipeline of a wave's steps: page ids two steps ahead, K and V one.  Lane i (mod 8)
  // looks up the page of group i (mod groups) of 8 tokens (a group never crosses a page).
  constexpr int kGroups = S::kTokens / 8, kStride = S::kTokens * kWaves;
  uint8_t* mine = lds + wave * S::kLds;
  S step;
  int id, page;                                // of the step after the one being loaded
  auto look_up = [&](int t) {
    const int tok = t + 8 * (lane % kGroups);
    page = (int)((((uint32_t)tok >> 3) * p.page_magic) >> 36);
    id = tok < end ? table[page] : -1;
  };
  uint32_t held = 0, next_held = 0;            // bit i: group i's page is held
  uint32_t row8 = 0;
  auto load = [&](int t) {
    const bool in = (uint32_t)id < (uint32_t)a.c.num_pages;
    // rows of the cache in groups of 8 (fewer than 2^32); where no page is held row 0 is
    // read and masked
    const int off = t + 8 * (lane % kGroups) - page * a.c.page_size;
    row8 = in ? ((uint32_t)id * a.c.heads + head) * ((uint32_t)a.c.page_size >> 3) +
                               ((uint32_t)off >> 3) : 0u;
    next_held = (uint32_t)__ballot(in);
    step.load(a.c, row8, lane);
  };
  int t = begin + S::kTokens * wave;
  look_up(t);
  const uint16_t* qrow = a.q + run.b * a.q_stride + (int64_t)(head * a.G + g0 + r) * D;
  u32x4 raw[kSteps];
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
  }
  if (t < end) {
    load(t);
    step.load_late(a.c, row8, lane);
    look_up(t + kStride);
  }

  // Queries: column r of both products, scaled by a power of two that goes into the scale
  // of the scores.  Beside a bf16 cache they are bf16 and only ever scaled up, to a largest of
  // 1 or more, which loses nothing; beside an NVFP4 one half precision, the largest in [2^14,
  // 2^15): exact for bf16 values down to 2^-31 of it.  A wave that holds a smaller one (K may
  // be 0 beside the large ones, so that it decides the scores) takes the queries as bf16 there
  // too (every wave of 16 x up to 32768 tokens: 66.4 us instead of 64.3).
  u32x4 qf[kSteps];
  float cs;
  bool in_bf16 = false;
  {
    uint32_t mx = 0, least = ~0u;              // least: of the magnitudes but 0, less 1
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      mx = pk_max_abs4(mx, make_uint4(raw[j].x, raw[j].y, raw[j].z, raw[j].w));
      if constexpr (kNVFP4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) least = pk_min_less1(least, raw[j][i]);
      }
    }
    const float top = max_over_groups(__uint_as_float(pk_max_to_f32_bits(mx)));
    int e = top > 0.0f ? ilogbf(top) : 0;      // queries times 2^-e
    int more = 0;                              // K times 2^-more
    if constexpr (kNVFP4) {
      const int field = (int)((min(least & 0xffffu, least >> 16) + 1) >> 7);
      in_bf16 = __any(field < e + 127 - 31);
      e = in_bf16 ? min(e, 0) : e - 14;
      more = in_bf16 ? kShiftBf16 : 0;
    } else {
      e = min(e, 0);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = ldexpf(bf16_lo(raw[j][i]), -e), y = ldexpf(bf16_hi(raw[j][i]), -e);
        qf[j][i] = kNVFP4 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
      }
    if (kNVFP4 && in_bf16) {
      asm volatile("");                        // a branch, not selects for every query
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[j][i] = pack_bf16x2(ldexpf(bf16_lo(raw[j][i]), -e), ldexpf(bf16_hi(raw[j][i]), -e));
    }
    // the sign of the scale goes into the queries: cs >= 0, and the maximum can be taken
    // before the scale (a scale of 0 as queries of 0: -inf * 0 is not -inf)
    const float full = ldexpf(a.scale * kLog2e * kt0, e + more);
    cs = full == 0.0f ? 1.0f : fabsf(full) > FLT_MAX ? FLT_MAX : fabsf(full);   // inf * 0 is not 0
    if (!(full > 0.0f)) {
      const uint32_t flip = full < 0.0f ? 0x80008000u : 0u, keep = full < 0.0f ? ~0u : 0u;
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[j][i] = (qf[j][i] & keep) ^ flip;
    }
  }

  f32x4 o[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) o[i] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;

  for (; t < end; t += kStride) {
    step.stage(mine, lane);
    held = next_held;
    if (t + kStride < end) {
      load(t + kStride);
      look_up(t + 2 * kStride);
    }
    uint32_t seen[N];                          // bit e: token e of the lane's 8 is visible
    bool all = true;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int tok = t + 32 * n + 8 * q;      // visible: tokens first .. end - 1 of the 8
      const int lo = min(max(rg.first - tok, 0), 8), hi = min(max(end - tok, 0), 8);
      seen[n] = (held >> (4 * n + q)) & 1 ? (0xffu >> (8 - hi)) & (0xffu << lo) & 0xffu : 0u;
      all = all && seen[n] == 0xffu;
    }
    all = __all(all);

    if (!all) {
      asm volatile("");                        // a branch, not selects in every step
      step.mask_v(mine, seen, lane);
    }
    if constexpr (kNVFP4) step.read_all(mine, r, q);
    float w[N][8];                             // scores, before cs
    if (!kNVFP4 || !in_bf16) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 s = step.scores(mine, qf, n, u, r, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[n][4 * u + i] = s[i];
        }
    } else if constexpr (kNVFP4) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 s = step.scores_bf16(qf, n, u);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[n][4 * u + i] = s[i];
        }
    }
    if (!all) {
      asm volatile("");
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) w[n][e] = (seen[n] >> e) & 1 ? w[n][e] : -INFINITY;
    }
    // Rescaling.  m is a common reference of a head's four lanes rather than the exact
    // maximum: it moves only when a score is more than 2^kSlack above where it was set, so
    // that most steps need neither the exchange between the lanes nor the products with o.
    // It is set to 2^kBelow under the maximum: the largest weight is between 2^kBelow and
    // 2^(kBelow + kSlack), inside half precision, whose 11 bits reach down to 2^-21 of it or
    // less and whose last step is 2^-32 of it (from 1 on up they would reach 2^-14 and 2^-25).
    float top = w[0][0];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, w[n][e]);
    top *= cs;
    if (__any(top > m + (kBelow + kSlack))) {
      const float m2 = fmaxf(m, max_over_groups(top) - kBelow);
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
#pragma unroll
    for (int n = 0; n < N; ++n) {
      u32x4 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(w[n][e], cs, -m0));
        l += w[n][e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = w[n][2 * e], y = w[n][2 * e + 1];
        if constexpr (kNVFP4) {
          hi[e] = pack_f16x2(x, y);
        } else {
          hi[e] = pack_bf16x2(x, y);
          lo[e] = pack_bf16x2(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
        }
      }
      step.accumulate(mine, o, n, hi, lo, r, q);
    }
    if (t + kStride < end) step.load_late(a.c, row8, lane);
  }
  __syncthreads();                             // the pieces of LDS take the waves' o

  // join the waves
  l = sum_over_groups(l);
  if (q == 0) {
    sm[wave][r] = m;
    sl[wave][r] = l;
  }
  float(*so)[kHeads][kPad] = reinterpret_cast<float(*)[kHeads][kPad]>(lds);
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
  float* parts = p.parts + ((int64_t)hg * (p.runs + a.B) + run.b) * part_stride(p);
  float* part = parts + (int64_t)(blockIdx.x / per) * part_stride(p);
  const int64_t hrow0 = (int64_t)run.b * a.Hq + head * a.G + g0;
  int tid = threadIdx.x;
  asm("" : "+v"(tid));       // what depends on it is not to be kept through the steps
  for (int i = tid; i < rows * (D / 2); i += kThreads) {
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
    if (whole) {
      const float n = ll == 0.0f ? 0.0f : vt0 / ll;
      *reinterpret_cast<uint32_t*>(a.out + (hrow0 + g) * D + d) = pack_bf16x2(x * n, y * n);
      if (d == 0 && a.lse) a.lse[hrow0 + g] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    } else {
      store_shared(part + g * D + d, f32x2{x, y});
      if (d == 0) store_shared(part + p.rows * D + 2 * g, f32x2{mm, ll});
    }
  }
  if (!whole) {
    int first = run.first, count = run.count;
    if (!run.one) {
      first = scalar((uint32_t)run.at / (uint32_t)run.share);
      count = scalar((uint32_t)(run.at + run.steps - 1) / (uint32_t)run.share) - first + 1;
    }
    const Joining j = plan_joining<D>(rows, count);
    const float* src = parts + first * part_stride(p);
    uint32_t* arrived = p.arrived + (int64_t)run.b * per + hg;
    uint32_t* counter = arrived;
    float* to = nullptr;
    int n = count;
    // Group k has counter and result first + 1 + k of the head group's runs: there are
    // fewer groups than runs between the first and the last, which are this sequence's.
    const int at = hg * p.runs + first + 1;
    if (j.groups > 1) {
      const int k = scalar((uint32_t)(blockIdx.x / per - first) / (uint32_t)j.size);
      n = min(j.size, count - k * j.size);
      src += k * j.size * part_stride(p);
      to = p.group_parts + (at + k) * part_stride(p);
      counter = p.grouped + at + k;
    }
    while (last_to_finish(counter, n, before_me)) {
      join_partials<D>(p, src, n, j.split, rows, to, hrow0, vt0, reinterpret_cast<Joined*>(lds));
      reset_counter(counter);
      if (!to) break;
      n = j.groups;
      src = p.group_parts + at * part_stride(p);
      to = nullptr;
      counter = arrived;
    }
  }
  run.pos += steps;
  }
}

// `steps`: of one head at most, by the table's capacity.
template <bool kNVFP4, int D>
void launch(Plan& p, int64_t steps, hipStream_t s) {
  const int per = p.a.c.heads * p.groups;
  p.runs = (int)max(min((int64_t)(kPerCU<D> * kCUs / per), steps), (int64_t)1);
  p.group_parts = p.parts + (int64_t)per * (p.runs + p.a.B) * part_floats(p.rows, D);
  paged_decode_kernel<kNVFP4, D><<<(uint32_t)(p.runs * per), kThreads, 0, s>>>(p);
}
template <bool kNVFP4>
void launch_dim(Plan& p, int64_t steps, hipStream_t s) {
  switch (p.a.c.dim) {
    case 32: return launch<kNVFP4, 32>(p, steps, s);
    case 64: return launch<kNVFP4, 64>(p, steps, s);
    case 96: return launch<kNVFP4, 96>(p, steps, s);
    case 128: return launch<kNVFP4, 128>(p, steps, s);
    case 160: return launch<kNVFP4, 160>(p, steps, s);
    case 192: return launch<kNVFP4, 192>(p, steps, s);
    case 224: return launch<kNVFP4, 224>(p, steps, s);
    default: return launch<kNVFP4, 256>(p, steps, s);
  }
}

// Segments of one sequence, and the sequences of one launch.
int64_t segments_of(int64_t Hq, int64_t heads) {
  return heads * ((Hq / heads + kHeads - 1) / kHeads);
}
int64_t launch_seqs(int64_t B, int64_t per) { return min(B, kCounters / per); }

}  // namespace

bool decode_heads_ok(int64_t Hq, int64_t heads) { return segments_of(Hq, heads) <= kCounters; }

size_t decode_workspace_bytes(int64_t B, int64_t Hq, int64_t heads, int64_t dim) {
  const int64_t G = Hq / heads, per = segments_of(Hq, heads);
  const int64_t runs = max(kMaxResident / per, (int64_t)1);
  const int64_t parts = (runs + launch_seqs(B, per)) * per + runs * per;
  return kCounterBytes +
         sizeof(float) * (size_t)(parts * part_floats(G < kHeads ? (int)G : kHeads, (int)dim));
}

hipError_t launch_paged_decode(const DecodeArgs& args, hipStream_t s) {
  Plan p;
  p.a = args;
  const DecodeArgs& a = p.a;
  p.groups = (a.G + kHeads - 1) / kHeads;
  p.rows = a.G < kHeads ? a.G : kHeads;
  const uint64_t d = a.c.page_size / 8;
  p.page_magic = (((uint64_t)1 << 36) + d - 1) / d;
  p.arrived = static_cast<uint32_t*>(a.ws);
  p.grouped = p.arrived + kCounters;
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kCounterBytes);
  const int64_t per = (int64_t)a.c.heads * p.groups, B = args.B, seqs = launch_seqs(B, per);
  for (int64_t b = 0; b < B; b += seqs) {
    p.a.B = (int)min(seqs, B - b);
    p.a.q = args.q + b * args.q_stride;
    p.a.table = args.table + b * args.table_stride;
    p.a.lens = args.lens + b;
    p.a.out = args.out + b * args.Hq * args.c.dim;
    p.a.lse = args.lse ? args.lse + b * args.Hq : nullptr;
    // the table's capacity bounds the steps (a visible range starts at a multiple of 8
    // tokens, so it never takes a step more)
    const int64_t cap = (int64_t)a.pages_per_seq * a.c.page_size;
    const int64_t steps = p.a.B * max((cap + kStepTokens - 1) / kStepTokens, (int64_t)1);
    if (a.c.nvfp4) launch_dim<true>(p, steps, s);
    else launch_dim<false>(p, steps, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fos
