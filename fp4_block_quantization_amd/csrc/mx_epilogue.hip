// Products of MXFP4 records with an epilogue: Y = act(deq(A) deq(B)^T + bias) + residual, or
// gated, on the scaled FP4 matrix cores (v_mfma_scale_f32_32x32x64_f8f6f4, both operands
// E2M1), which take the packed bytes and E8M0 scales as they are.  Sums are taken in
// the order of fos_mx_qlinear_fwd's, but for the tiles that split K.
//
// A workgroup has a (64 TI) x (64 TJ) tile, TI x TJ MFMA tiles to a wave.  K in stages
// of 128 (64 bytes of nibbles a row), NS of them in LDS: four, or two where two workgroups of
// 256 x 128 share a CU.  The E8M0 bytes of four stages (16 a row) are copied at once, apart,
// and go to registers: a row's scale bytes of one stage are a request of their own to the
// address unit, as dear as 64 bytes of nibbles.  The copies are what bounds the kernel: the
// matrix cores are busy 43% of the time, VALU 17 to 24% (4096 x 12288 x 4096 gated with silu
// 233 to 238 us, 3.5 PFLOP/s; two stages of 256 with their scales beside them: 257 where
// this took 244).
//
// A stage is two k-steps of 64.  While one multiplies, the operands of the next are read from
// LDS; between the two stands the stage's one barrier, where every wave has read all of this
// stage (the NS-th stage after it is copied to its place at once) and the next one has
// landed (it had NS - 1 stages' time).
#include "feedforward.hpp"
#include "gemm_common.hpp"
#include "gemm_epilogue.hpp"

namespace fos {

namespace {

using namespace gemm;

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStageK = 128;
constexpr int kStageRowBytes = kStageK / 2;
constexpr int kScaleStages = 4;                                    // stages of one scale copy
constexpr int kScaleRowBytes = kScaleStages * kStageK / 32;        // 16

template <int TI, int TJ>
struct FlowStage {
  uint8_t a[64 * TI * kStageRowBytes];
  uint8_t b[64 * TJ * kStageRowBytes];
};
template <int TI, int TJ>
struct FlowScales {
  uint8_t a[64 * TI * kScaleRowBytes];
  uint8_t b[64 * TJ * kScaleRowBytes];
};

struct FlowOperands {
  __amdgpu_buffer_rsrc_t a, sa, b, sb;
  uint32_t oa, osa, osb;      // per-lane offsets
  uint32_t ob[2];             // with a gate, TJ = 4: of each projection's rows
  uint32_t group_stride;      // bytes between row-groups (16 rows)
};

// Copies of one wave, the same number for each: a quarter of a stage's rows, 16 rows to an
// instruction, and 64 rows' scales of each operand (where there are fewer of them than waves,
// two copy the same).
template <int TI, int TJ, bool kGate>
__device__ __forceinline__ void flow_load(FlowStage<TI, TJ>& st, const FlowOperands& p, int s, int wave) {
  const int od = s * kStageRowBytes;
#pragma unroll
  for (int q = 0; q < TI; ++q)
    dma16(p.a, st.a + (16 * TI * wave + 16 * q) * kStageRowBytes, p.oa, od + q * (int)p.group_stride);
#pragma unroll
  for (int q = 0; q < TJ; ++q) {
    const bool up = kGate && TJ == 4 && q >= 2;
    dma16(p.b, st.b + (16 * TJ * wave + 16 * q) * kStageRowBytes, p.ob[up],
          od + (up ? q - 2 : q) * (int)p.group_stride);
  }
}
template <int TI, int TJ>
__device__ __forceinline__ void flow_load_scales(FlowScales<TI, TJ>& sc, const FlowOperands& p, int c,
                                                 int wave) {
  dma16(p.sa, sc.a + 64 * (wave % TI) * kScaleRowBytes, p.osa, c * kScaleRowBytes);
  dma16(p.sb, sc.b + 64 * (wave % TJ) * kScaleRowBytes, p.osb, c * kScaleRowBytes);
}

// Granule g (16 bytes, 32 values) of a row of a stage lies at g ^ ((row >> 2) & 3): 16 rows of
// an operand are read from different banks.
template <int T>
__device__ __forceinline__ void flow_operands(const uint8_t* base, int row, int g, i32x8 (&o)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(base + (row + 32 * i) * kStageRowBytes +
                                                    ((g ^ ((row >> 2) & 3)) << 4));
    o[i] = i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  }
}
template <int T>
__device__ __forceinline__ void flow_scales(const uint8_t* base, int row, uint4 (&s)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i)
    s[i] = *reinterpret_cast<const uint4*>(base + (row + 32 * i) * kScaleRowBytes);
}
__device__ __forceinline__ uint32_t scale_word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// Byte kByte of the scale words.
template <int kByte, int TI, int TJ>
__device__ __forceinline__ void flow_mma(const i32x8 (&A)[TI], const i32x8 (&B)[TJ],
                                         const int (&xa)[TI], const int (&xb)[TJ],
                                         f32x16 (&acc)[TI][TJ]) {
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int n = 0; n < TJ; ++n)
      acc[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A[i], B[n], acc[i][n], 4, 4,
                                                                   kByte, xa[i], kByte, xb[n]);
}

// What stands before it is issued before what stands behind it.
__device__ __forceinline__ void flow_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// A workgroup barrier behind a wait for all but the newest kCopies copies of the wave and for
// all its LDS reads (__syncthreads would wait for every copy).
template <int kCopies>
__device__ __forceinline__ void flow_barrier() {
  static_assert(kCopies < 64, "the counter's range");
  flow_order();
  __builtin_amdgcn_s_waitcnt((kCopies & 15) | 7 << 4 | (kCopies >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// The order of a phase: one MFMA, then an LDS read and a copy while there are some.
template <int kMfmas, int kReads, int kCopies>
__device__ __forceinline__ void flow_schedule() {
  constexpr int kReadStep = (kReads + kMfmas - 1) / kMfmas, kCopyStep = (kCopies + kMfmas - 1) / kMfmas;
#pragma unroll
  for (int m = 0; m < kMfmas; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (m * kReadStep < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kReadStep, 0);
    if (m * kCopyStep < kCopies) __builtin_amdgcn_sched_group_barrier(0x020, kCopyStep, 0);
  }
}

template <int J, typename T>
__device__ __forceinline__ T& pick(T& a, T& b, T& c, T& d) {
  if constexpr (J == 0) return a;
  if constexpr (J == 1) return b;
  if constexpr (J == 2) return c;
  return d;
}

// Copies are counted from the newest.  Phase p (of four, again and again) issues, behind stage p's
// barrier, the data copies of stage p + NS, and phase 0 those of the scales too, which the read in
// phase 3 takes.  Within a phase they may be issued in any order: they go to different objects
// and share scheduling groups.  So only whole phases count as on their way at stage J's barrier,
// those after the phase of stage J + 1's copies.
constexpr int kScaleCopies = 2;
constexpr int flow_in_flight(int ns, int copies, int j) {
  int n = 0;
  for (int p = j + 2 - ns; p < j; ++p) n += copies + (p == 0 ? kScaleCopies : 0);
  return n;
}
// Whether with these counts everything has landed that is read behind a barrier, whichever way
// the copies of phase 0 are ordered: two rounds of four stages played through.
constexpr bool flow_lands(int ns, int copies, bool scales_first) {
  constexpr int kRounds = 2, kStages = 4 * kRounds;
  int data_end[kStages + 4] = {}, scales_end[kRounds] = {}, issued = ns * copies;
  for (int s = 0; s < ns; ++s) data_end[s] = (s + 1) * copies;
  for (int s = 0; s < kStages; ++s) {
    const int landed = issued - flow_in_flight(ns, copies, s % 4);
    if (data_end[s + 1] > landed || (s % 4 == 3 && scales_end[s / 4] > landed)) return false;
    if (s % 4 == 0 && scales_first) scales_end[s / 4] = issued += kScaleCopies;
    data_end[s + ns] = issued += copies;
    if (s % 4 == 0 && !scales_first) scales_end[s / 4] = issued += kScaleCopies;
  }
  return true;
}

// The products of this wave's tiles.  With kSplit > 1 a group of four waves has every
// kSplit-th four stages, all groups as many: those past the last count with scales of 2^-127,
// whose products are 0 in fp32.
template <int TI, int TJ, int NS, bool kGate, int kSplit>
__device__ __forceinline__ void flow_products(FlowStage<TI, TJ>& st0, FlowStage<TI, TJ>& st1,
                                              FlowStage<TI, TJ>& st2, FlowStage<TI, TJ>& st3,
                                              FlowScales<TI, TJ>& sc, const FlowOperands& p,
                                              f32x16 (&acc)[TI][TJ], int ra, int rb, int h,
                                              int wave, int stages, int group) {
  static_assert(NS == 2 || NS == 4, "stages take turns within four");
  constexpr int kMfmas = TI * TJ, kReads = TI + TJ, kCopies = TI + TJ;
  static_assert(flow_lands(NS, kCopies, false) && flow_lands(NS, kCopies, true),
                "a barrier waits for what is read behind it");
  // the stage behind the group's s-th
  auto at = [&](int s) { return kSplit == 1 ? s : (s & ~3) * kSplit + 4 * group + (s & 3); };
  // what is copied past the last stage is the last one again
  auto load = [&](FlowStage<TI, TJ>& st, int s) {
    flow_load<TI, TJ, kGate>(st, p, min(at(s), stages - 1), wave);
  };
  flow_load_scales(sc, p, at(0) / 4, wave);
  load(st0, 0);
  flow_order();   // the barriers' counts take the stages' copies in their order
  load(st1, 1);
  if constexpr (NS == 4) {
    flow_order();
    load(st2, 2);
    flow_order();
    load(st3, 3);
  }
  flow_barrier<(NS - 1) * kCopies>();
  uint4 sa[TI], sb[TJ];
  i32x8 A[TI], B[TJ], An[TI], Bn[TJ];
  flow_scales(sc.a, ra, sa);
  flow_scales(sc.b, rb, sb);
  flow_operands(st0.a, ra, h, A);
  flow_operands(st0.b, rb, h, B);

  // Stage S, the J-th of its four.
#define FOS_FLOW_STAGE(S, J)                                                                        \
  {                                                                                                 \
    FlowStage<TI, TJ>& cur = pick<(J) % NS>(st0, st1, st2, st3);                                    \
    FlowStage<TI, TJ>& next = pick<((J) + 1) % NS>(st0, st1, st2, st3);                             \
    int xa[TI], xb[TJ];                                                                             \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) xa[i] = (int)(scale_word(sa[i], J) >> (8 * h));  \
    _Pragma("unroll") for (int i = 0; i < TJ; ++i) xb[i] = (int)(scale_word(sb[i], J) >> (8 * h));  \
    if (kSplit > 1 && at(S) >= stages) {                                                            \
      _Pragma("unroll") for (int i = 0; i < TI; ++i) xa[i] = 0;                                     \
      _Pragma("unroll") for (int i = 0; i < TJ; ++i) xb[i] = 0;                                     \
    }                                                                                               \
    flow_operands(cur.a, ra, 2 + h, An);                                                            \
    flow_operands(cur.b, rb, 2 + h, Bn);                                                            \
    flow_mma<0>(A, B, xa, xb, acc);                                                                 \
    flow_schedule<kMfmas, kReads, 0>();                                                             \
    flow_barrier<flow_in_flight(NS, kCopies, J)>();                                                 \
    load(cur, (S) + NS);                                                                            \
    if (J == 0) flow_load_scales(sc, p, at((S) + 4) / 4, wave);                                     \
    if (J == 3) {                                                                                   \
      flow_scales(sc.a, ra, sa);                                                                    \
      flow_scales(sc.b, rb, sb);                                                                    \
    }                                                                                               \
    flow_operands(next.a, ra, h, A);                                                                \
    flow_operands(next.b, rb, h, B);                                                                \
    flow_mma<2>(An, Bn, xa, xb, acc);                                                               \
    flow_schedule<kMfmas, kReads + (J == 3 ? kReads : 0), kCopies + (J == 0 ? kScaleCopies : 0)>(); \
    __builtin_amdgcn_sched_barrier(0);                                                              \
  }
  if constexpr (kSplit > 1) {
    for (int s = 0; s < (stages + 4 * kSplit - 1) / (4 * kSplit) * 4; s += 4) {
      FOS_FLOW_STAGE(s, 0)
      FOS_FLOW_STAGE(s + 1, 1)
      FOS_FLOW_STAGE(s + 2, 2)
      FOS_FLOW_STAGE(s + 3, 3)
    }
  } else {
    int s = 0;
    for (; s + 3 < stages; s += 4) {
      FOS_FLOW_STAGE(s, 0)
      FOS_FLOW_STAGE(s + 1, 1)
      FOS_FLOW_STAGE(s + 2, 2)
      FOS_FLOW_STAGE(s + 3, 3)
    }
    if (s < stages) {   // K % 256 == 0: two stages
      FOS_FLOW_STAGE(s, 0)
      FOS_FLOW_STAGE(s + 1, 1)
    }
  }
#undef FOS_FLOW_STAGE
}

constexpr int flow_waves_per_simd(int mfma_tiles, int split) {
  return mfma_tiles == 16 ? 1 : split == 4 ? 4 : 2;
}

// With kSplit = 4 four groups of four waves share a tile of 64 x 64, for so few tiles that
// each has a CU of its own.
template <int TI, int TJ, int NS, int kEpi, int kSplit>
__global__ __attribute__((amdgpu_flat_work_group_size(256 * kSplit, 256 * kSplit),
                          amdgpu_waves_per_eu(flow_waves_per_simd(TI * TJ, kSplit),
                                              flow_waves_per_simd(TI * TJ, kSplit))))
void mx_flow_kernel(const uint8_t* __restrict__ ad, const uint8_t* __restrict__ as,
                    const uint8_t* __restrict__ bd, const uint8_t* __restrict__ bs, int M, int N,
                    int K, int tiles_m, int tiles_n, void* __restrict__ y, EpilogueArgs e) {
  constexpr bool kGate = kEpi == kGated;
  constexpr int kProj = kGate ? 2 : 1;   // weight rows of one column of Y
  constexpr int kBM = 64 * TI, kBN = 64 * TJ;
  // objects of their own: the compiler then knows that a copy to one does not touch another
  __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st0;
  __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st1;
  __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st2;
  __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st3;
  __shared__ __attribute__((aligned(16))) FlowScales<TI, TJ> sc;
  const TileCoord tc = tile_of(blockIdx.x, tiles_m, tiles_n);
  const int tm = tc.tm, tn = tc.tn;
  const int lane = threadIdx.x & 63;
  const int group = kSplit == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) - 4 * group;
  const int lr = lane & 31, h = lane >> 5;
  const uint32_t kb2 = K / 2, kb32 = K / 32;
  const int ra = (wave >> 1) * (32 * TI) + lr;
  const int rb = (wave & 1) * (32 * TJ) + lr;
  const int stages = K / kStageK;

  FlowOperands p;
  p.a = __builtin_amdgcn_make_buffer_rsrc((void*)ad, 0, (int)((uint32_t)M * kb2), kRsrcWord3);
  p.sa = __builtin_amdgcn_make_buffer_rsrc((void*)as, 0, (int)((uint32_t)M * kb32), kRsrcWord3);
  p.b = __builtin_amdgcn_make_buffer_rsrc((void*)bd, 0, (int)((uint32_t)(kProj * N) * kb2), kRsrcWord3);
  p.sb = __builtin_amdgcn_make_buffer_rsrc((void*)bs, 0, (int)((uint32_t)(kProj * N) * kb32), kRsrcWord3);
  p.group_stride = 16 * kb2;
  // the weight row behind row r of the tile
  auto weight_row = [&](int r) -> uint32_t {
    if constexpr (!kGate) return tn * kBN + r;
    bool up;
    const int g = gated_row(r, up);
    return tn * (kBN / 2) + g + (up ? N : 0);
  };
  {
    // lane l of row-group q writes LDS slot (l & 3) of local row kBM/4*wave + 16*q + (l >> 2),
    // and fetches the granule that belongs there
    const uint32_t sub = lane >> 2, g = (lane & 3) ^ ((lane >> 4) & 3);
    p.oa = (uint32_t)(tm * kBM + 16 * TI * wave + sub) * kb2 + 16 * g;
    p.ob[0] = weight_row(16 * TJ * wave + sub) * kb2 + 16 * g;
    p.ob[1] = p.ob[0] + (uint32_t)N * kb2;
    p.osa = (uint32_t)(tm * kBM + 64 * (wave % TI) + lane) * kb32;
    p.osb = weight_row(64 * (wave % TJ) + lane) * kb32;
  }

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int n = 0; n < TJ; ++n) acc[i][n] = f32x16{};

  if constexpr (kSplit == 1) {
    flow_products<TI, TJ, NS, kGate, 1>(st0, st1, st2, st3, sc, p, acc, ra, rb, h, wave, stages, 0);
    __builtin_amdgcn_s_waitcnt(0);   // no copy outlives the workgroup
    store_fused<TI, TJ, kGate>(e, y, M, N, tm * kBM + (wave >> 1) * (32 * TI),
                               (tn * kBN + (wave & 1) * (32 * TJ)) / kProj, lane, 1.0f, acc);
  } else {
    static_assert(kSplit == 4 && TI == 1 && TJ == 1 && NS == 4, "one tile to a wave, joined");
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st4;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st5;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st6;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st7;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st8;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st9;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st10;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st11;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st12;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st13;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st14;
    __shared__ __attribute__((aligned(16))) FlowStage<TI, TJ> st15;
    __shared__ __attribute__((aligned(16))) FlowScales<TI, TJ> sc1;
    __shared__ __attribute__((aligned(16))) FlowScales<TI, TJ> sc2;
    __shared__ __attribute__((aligned(16))) FlowScales<TI, TJ> sc3;
    if (group == 0)
      flow_products<TI, TJ, NS, kGate, 4>(st0, st1, st2, st3, sc, p, acc, ra, rb, h, wave, stages, 0);
    else if (group == 1)
      flow_products<TI, TJ, NS, kGate, 4>(st4, st5, st6, st7, sc1, p, acc, ra, rb, h, wave, stages, 1);
    else if (group == 2)
      flow_products<TI, TJ, NS, kGate, 4>(st8, st9, st10, st11, sc2, p, acc, ra, rb, h, wave, stages, 2);
    else
      flow_products<TI, TJ, NS, kGate, 4>(st12, st13, st14, st15, sc3, p, acc, ra, rb, h, wave, stages, 3);
    __builtin_amdgcn_s_waitcnt(0);   // no copy is on its way to where the sums go
    static_assert(kJoinBytes == 2 * sizeof(FlowStage<TI, TJ>), "the sums take two stages' place");
    store_joined<kGate>(e, y, M, N, tm, tn, wave, wave, group, lane, 1.0f, acc[0][0], [&](int g, int half) {
      return g == 0 ? (half ? st1 : st0).a : g == 1 ? (half ? st5 : st4).a
           : g == 2 ? (half ? st9 : st8).a : (half ? st13 : st12).a;
    });
  }
}

template <int TI, int TJ, int NS, int kEpi, int kSplit = 1>
hipError_t launch_flow(const QLinearArgs& a, hipStream_t s) {
  constexpr int kCols = 64 * TJ / (kEpi == kGated ? 2 : 1);
  const int tiles_m = (int)((a.M + 64 * TI - 1) / (64 * TI));
  const int tiles_n = (int)((a.N + kCols - 1) / kCols);
  mx_flow_kernel<TI, TJ, NS, kEpi, kSplit><<<tiles_m * tiles_n, 256 * kSplit, 0, s>>>(
      a.xd, a.xs, a.wd, a.ws, (int)a.M, (int)a.N, (int)a.K, tiles_m, tiles_n, a.y, a.e);
  return hipGetLastError();
}

// Kernel of an epilogue's product, by what a round of workgroups takes (us, measured with
// silu: fixed, and per 4096 of K): 64 x 64 tiles with K split over four groups of waves, while
// every tile has a CU of its own; 128 x 128 tiles, two to a CU or (half a round) one, while
// there are few; 256 x 128, whose epilogues run beside another workgroup's products, for a
// short K; 256 x 256, which copies least for its products, for a long one.  In this order:
// 16 x 4096 x 4096 8.9, 11.0, - and 17; 64 x 4096 x 12288 18, 23, - and 37 with the weight in a
// cache (23 with the first from memory); 1024 x 4096 x 4096 -, 19, 24 and 36; 8192 x 8192 x 1024
// -, 70, 64 and 86; 4096 x 4096 x 12288 -, 155, 126 and 108.  (All measured with an earlier epilogue;
// the chosen ones now take 8.5, 17, 17, 62 and 104.)
struct MxShape {
  int ti, tj, split, resident;
  float half, half_k, full, full_k;
};
constexpr MxShape kMxShapes[] = {{1, 1, 4, 256, 5.5f, 4.8f, 6.0f, 5.6f},
                                 {2, 2, 1, 512, 6.0f, 12.4f, 5.0f, 24.0f},
                                 {4, 2, 1, 512, 8.0f, 21.0f, 7.0f, 38.5f},
                                 {4, 4, 1, 256, 14.0f, 29.7f, 14.0f, 29.7f}};
int64_t mx_tiles(const QLinearArgs& a, const MxShape& h) {
  const int64_t cols = a.gated ? 32 * h.tj : 64 * h.tj;
  return ((a.M + 64 * h.ti - 1) / (64 * h.ti)) * ((a.N + cols - 1) / cols);
}
const MxShape& mx_shape(const QLinearArgs& a) {
  const MxShape* best = nullptr;
  float least = 0.0f;
  const float k = (float)a.K / 4096.0f;
  for (const MxShape& h : kMxShapes) {
    const int64_t tiles = mx_tiles(a, h), full = tiles / h.resident, rest = tiles % h.resident;
    // no second four stages to split, or more than one round
    if (h.split > 1 && (a.K <= 4 * kStageK || tiles > h.resident)) continue;
    float us = (float)full * (h.full + h.full_k * k);
    if (rest) us += 2 * rest <= h.resident ? h.half + h.half_k * k : h.full + h.full_k * k;
    if (!best || us < least) {
      best = &h;
      least = us;
    }
  }
  return *best;
}

template <int kEpi>
hipError_t launch_mx_epi(const QLinearArgs& a, hipStream_t s) {
  const MxShape& h = mx_shape(a);
  if (h.split == 4) return launch_flow<1, 1, 4, kEpi, 4>(a, s);
  if (h.tj == 4) return launch_flow<4, 4, 4, kEpi>(a, s);
  if (h.ti == 4) return launch_flow<4, 2, 2, kEpi>(a, s);
  return launch_flow<2, 2, 4, kEpi>(a, s);
}

}  // namespace

int64_t mx_epilogue_grid(const QLinearArgs& a) { return mx_tiles(a, mx_shape(a)); }

hipError_t launch_mx_epilogue(const QLinearArgs& a, hipStream_t s) {
  return a.gated ? launch_mx_epi<kGated>(a, s) : launch_mx_epi<kFused>(a, s);
}

}  // namespace fos
