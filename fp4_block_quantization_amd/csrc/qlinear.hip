// Simulated quantized linear forward, Y = deq(Xq) . deq(Wq)^T (Four Over Six
// documentation page, section "Four Over Six": where native FP4 matrix operations
// are missing, the quantized linear layer is simulated with a higher-precision
// matrix multiplication of the dequantized operands; Ultralytics glossary "FP4",
// section "FP4 for inference and training": FP4 products accumulate in higher
// precision).
//
// Every dequantized operand value E2M1 * E4M3 has at most 6 significant bits and
// lies in [2^-10, 2688], so it is exact in fp16; fp16 x fp16 products are exact in
// fp32.  The kernel therefore forms E*D in fp16 registers (hardware E2M1->f16 and
// E4M3->f16 conversions, one packed f16 multiply per pair) and feeds them straight to
// v_mfma_f32_32x32x16_f16 with fp32 accumulation; the tensor scales t_x * t_w are
// applied in fp32 in the epilogue, then the result is rounded to bf16.
//
// Tiling: a 256-thread workgroup owns a 256x256 tile of Y, each wave a 128x128
// quarter held as 4x4 MFMA accumulators (256 fp32 per lane).  Both operands are
// K-major, so a lane's 8 MFMA k-slots come from one 4-byte word of packed nibbles; A
// and B use the same k mapping, so the reordering of k inside a chunk cancels in the
// sum.  Two kernels:
//   qlinear_lds_kernel (K % 256 == 0): packed operands are copied global -> LDS in
//     256-wide K stages (double-buffered) and dequantized from LDS, software-pipelined
//     against the MFMAs;
//   qlinear_kernel (any K % 64 == 0): each wave reads its packed operands straight
//     from L2 into registers, three register stages deep.
// Workgroups are remapped so that each XCD (dispatched round-robin) runs a contiguous
// group of 4 tile-rows x all tile-columns.
//
// The LDS-staged kernel ends in a plain store or in the epilogue of gemm_epilogue.hpp (kEpi);
// with an epilogue it takes any K % 64 == 0 and, for few tiles, smaller ones.  With a gate,
// the weight rows of a tile are half the gate's and half those of the other projection that
// belong to the same columns of Y, 32 of each in turn: a wave has both factors of every
// product in its own accumulators.
#include "device_common.hpp"
#include "feedforward.hpp"
#include "gemm_common.hpp"
#include "gemm_epilogue.hpp"
#include "kernels.hpp"

namespace fos {

namespace {

using namespace gemm;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr int kChunk = 64;

__device__ __forceinline__ h8 dequant8(uint32_t w, h2 dd) {
  const h2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * dd;
  const h2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * dd;
  const h2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * dd;
  const h2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * dd;
  return h8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

__device__ __forceinline__ uint32_t word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// ---------------------------------------------------------------- register-staged kernel
// Packed operands of one 64-wide K chunk for one lane: 16 bytes of nibbles per A row
// tile and per B column tile, and the two E4M3 scale bytes that cover them.  Lane
// half h (lane / 32) takes the 32 consecutive k values [32h, 32h + 32) of the chunk
// in one 16-byte load per row, and k-step j uses word j of it.
template <int TI, int TJ>
struct Stage {
  uint4 a[TI], b[TJ];
  uint32_t sa[TI], sb[TJ];
};

// Operands are read through buffer resources (descriptor in SGPRs, 32-bit per-lane
// byte offsets): rows past M or N fall outside the resource and read as zero, and
// the per-chunk advance is a scalar offset.
template <int TI, int TJ>
struct Operands {
  __amdgpu_buffer_rsrc_t a, sa, b, sb;
  uint32_t oa[TI], osa[TI], ob[TJ], osb[TJ];
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint4 ld16(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff) {
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// The four scale bytes of a row's chunk are one aligned dword; lane half h uses
// bytes 2h and 2h + 1 (selected when the scales are converted).
template <int TI, int TJ>
__device__ __forceinline__ void load_stage(Stage<TI, TJ>& st, const Operands<TI, TJ>& p, int kc) {
  const int ob = kc * (kChunk / 2), os = kc * (kChunk / 16);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    st.a[i] = ld16(p.a, p.oa[i], ob);
    st.sa[i] = __builtin_amdgcn_raw_buffer_load_b32(p.sa, p.osa[i], os, 0);
  }
#pragma unroll
  for (int n = 0; n < TJ; ++n) {
    st.b[n] = ld16(p.b, p.ob[n], ob);
    st.sb[n] = __builtin_amdgcn_raw_buffer_load_b32(p.sb, p.osb[n], os, 0);
  }
}

template <int TI, int TJ>
__device__ __forceinline__ void mma_stage(const Stage<TI, TJ>& st, f32x16 (&acc)[TI][TJ],
                                          uint32_t sh) {
  h2 da[TI][2], db[TJ][2];
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const h2 sa = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st.sa[i] >> sh, 1.0f, false);
    da[i][0] = h2{sa.x, sa.x};
    da[i][1] = h2{sa.y, sa.y};
  }
#pragma unroll
  for (int n = 0; n < TJ; ++n) {
    const h2 sb = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(st.sb[n] >> sh, 1.0f, false);
    db[n][0] = h2{sb.x, sb.x};
    db[n][1] = h2{sb.y, sb.y};
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h8 A[TI], B[TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i) A[i] = dequant8(word(st.a[i], j), da[i][j >> 1]);
#pragma unroll
    for (int n = 0; n < TJ; ++n) B[n] = dequant8(word(st.b[n], j), db[n][j >> 1]);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int n = 0; n < TJ; ++n)
        acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[i], B[n], acc[i][n], 0, 0, 0);
  }
}

// Workgroup = 4 waves in a 2x2 arrangement; each wave owns TI x TJ MFMA tiles of
// 32x32, so the workgroup tile is (64*TI) x (64*TJ); WAVES_PER_EU waves share a SIMD.
template <int TI, int TJ, int STAGES, int WAVES_PER_EU>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256),
                          amdgpu_waves_per_eu(WAVES_PER_EU, WAVES_PER_EU)))
void qlinear_kernel(const uint8_t* __restrict__ xd, const uint8_t* __restrict__ xs,
                    const float* __restrict__ xt, const uint8_t* __restrict__ wd,
                    const uint8_t* __restrict__ ws, const float* __restrict__ wt, int M, int N,
                    int K, int tiles_m, int tiles_n, uint16_t* __restrict__ y) {
  constexpr int kWM = 32 * TI, kWN = 32 * TJ;     // wave tile
  constexpr int kBM = 2 * kWM, kBN = 2 * kWN;     // workgroup tile
  // ---- tile assignment: contiguous range per XCD, grouped along M inside it
  const TileCoord tc = tile_of(blockIdx.x, tiles_m, tiles_n);
  const int tm = tc.tm, tn = tc.tn;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 31, h = lane >> 5;
  const int m0 = tm * kBM + (wave >> 1) * kWM;
  const int n0 = tn * kBN + (wave & 1) * kWN;
  const uint32_t kb2 = K / 2, kb16 = K / 16;
  const uint32_t sh = 16 * h;   // this lane's scale byte pair within the dword

  Operands<TI, TJ> p;
  p.a = __builtin_amdgcn_make_buffer_rsrc((void*)xd, 0, (int)((uint32_t)M * kb2), kRsrcWord3);
  p.sa = __builtin_amdgcn_make_buffer_rsrc((void*)xs, 0, (int)((uint32_t)M * kb16), kRsrcWord3);
  p.b = __builtin_amdgcn_make_buffer_rsrc((void*)wd, 0, (int)((uint32_t)N * kb2), kRsrcWord3);
  p.sb = __builtin_amdgcn_make_buffer_rsrc((void*)ws, 0, (int)((uint32_t)N * kb16), kRsrcWord3);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const uint32_t r = m0 + 32 * i + lr;
    p.oa[i] = r * kb2 + 16 * h;
    p.osa[i] = r * kb16;
  }
#pragma unroll
  for (int n = 0; n < TJ; ++n) {
    const uint32_t c = n0 + 32 * n + lr;
    p.ob[n] = c * kb2 + 16 * h;
    p.osb[n] = c * kb16;
  }

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int n = 0; n < TJ; ++n) acc[i][n] = f32x16{};

  // register stages: chunk kc is multiplied while the next STAGES-1 chunks load
  const int nk = K / kChunk;
  Stage<TI, TJ> st[STAGES];
  int kc = 0;
  if (nk >= 2 * STAGES) {
    // unconditional prologue and a branch-free steady state, so the compiler can
    // wait on exactly the stage it consumes (any guarded load in or before the loop
    // makes it wait for every load instead); scheduling barriers keep each stage's
    // refill right after its last use (left alone, the scheduler sinks all refills
    // to the end of the loop body)
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      load_stage(st[s], p, s);
      __builtin_amdgcn_sched_barrier(0);   // keep stage order: stage 0 must be oldest
    }
    for (; kc + 2 * STAGES - 1 < nk; kc += STAGES) {
#pragma unroll
      for (int s = 0; s < STAGES; ++s) {
        mma_stage(st[s], acc, sh);
        __builtin_amdgcn_sched_barrier(0);
        load_stage(st[s], p, kc + s + STAGES);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
      if (s < nk) load_stage(st[s], p, s);
  }
  for (; kc < nk; kc += STAGES) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
      if (kc + s < nk) {
        mma_stage(st[s], acc, sh);
        if (kc + s + STAGES < nk) load_stage(st[s], p, kc + s + STAGES);
      }
    }
  }

  // ---- epilogue: lane (lr, h) holds, for accumulator element a, row
  // (a & 3) + 8 * (a >> 2) + 4 * h and column lr of each 32x32 tile.
  const float s = xt[0] * wt[0];
#pragma unroll
  for (int i = 0; i < TI; ++i) {
#pragma unroll
    for (int n = 0; n < TJ; ++n) {
      const int col = n0 + 32 * n + lr;
      if (col >= N) continue;
#pragma unroll
      for (int a = 0; a < 16; ++a) {
        const int row = m0 + 32 * i + (a & 3) + 8 * (a >> 2) + 4 * h;
        if (row < M) y[(int64_t)row * N + col] = (uint16_t)f32_to_bf16_rne(acc[i][n][a] * s);
      }
    }
  }
}

// ---------------------------------------------------------------- LDS-staged kernel
// K is consumed in super-chunks of 256 (128 bytes of nibbles and 16 scale bytes per
// row).  Each super-chunk of the workgroup's 256 A rows and 256 B rows is copied
// global -> LDS with buffer loads that write LDS directly (no VGPRs): a wave
// instruction moves 8 rows x 128 bytes, i.e. whole cache lines, so the L1 sees one
// request per line instead of one per 32-byte piece.  The 16-byte granules of a row
// are XOR-swizzled (slot = granule ^ ((row >> 1) & 7)) so that the per-lane
// ds_read_b128 of 16 consecutive rows hits distinct banks.  Two LDS stages of 72 KB:
// the next super-chunk is in flight while the current one is multiplied, with one
// workgroup barrier per super-chunk.
constexpr int kSuper = 256;                 // K per LDS stage
constexpr int kRowBytes = kSuper / 2;       // 128 bytes of nibbles per row per stage
constexpr int kRowScales = kSuper / 16;     // 16 scale bytes per row per stage
constexpr int kTileRows = 256;              // of the largest tile (TI = TJ = 4)

// Stage of a (64 TI) x (64 TJ) tile: 72 KB at 4 x 4.
template <int TI, int TJ>
struct LdsStage {
  uint8_t a[64 * TI * kRowBytes];
  uint8_t b[64 * TJ * kRowBytes];
  uint8_t sa[64 * TI * kRowScales];
  uint8_t sb[64 * TJ * kRowScales];
};

struct LdsOperands {
  __amdgpu_buffer_rsrc_t a, sa, b, sb;
  uint32_t oa[2], ob[2];      // per-lane offsets for even / odd row-groups
  uint32_t ou[2];             // with a gate, TJ = 4: of the other projection's rows
  uint32_t osa, osb;          // per-lane scale-row offsets
  uint32_t group_stride;      // bytes between row-groups (8 rows)
};

// The wave that copies the B scales of rows 64 u to 64 u + 63 has unit u; in smaller tiles
// these are the waves that copy no A scales.
template <int TJ>
__device__ __forceinline__ int b_scale_unit(int wave) {
  return TJ == 4 ? wave : 3 - wave;
}

// This wave's share of one super-chunk: a quarter of the rows of each operand in row-groups of
// 8 (one data instruction each), and 64 rows of scales (at 4 x 4 of both operands).
// Row-group q of the wave starts 8*q rows further on; the granule swizzle only depends on
// q's parity, so the per-lane offset is one of two values and the rest is a scalar offset.
// Part j copies row-group j of both operands, the last part the scale blocks.
template <int TI, int TJ>
constexpr int kLoadParts = 2 * (TI > TJ ? TI : TJ) + 1;
template <int TI, int TJ, bool kGate>
__device__ __forceinline__ void stage_load_part(LdsStage<TI, TJ>& st, const LdsOperands& p, int sc,
                                                int wave, int j) {
  if (j < kLoadParts<TI, TJ> - 1) {
    const int so = sc * kRowBytes + j * (int)p.group_stride;
    if (j < 2 * TI) dma16(p.a, st.a + (16 * TI * wave + 8 * j) * kRowBytes, p.oa[j & 1], so);
    // with a gate, row-groups 4 to 7 are the other projection's
    if (kGate && j >= 4)
      dma16(p.b, st.b + (16 * TJ * wave + 8 * j) * kRowBytes, p.ou[j & 1],
            sc * kRowBytes + (j - 4) * (int)p.group_stride);
    else if (j < 2 * TJ)
      dma16(p.b, st.b + (16 * TJ * wave + 8 * j) * kRowBytes, p.ob[j & 1], so);
  } else {
    const int os = sc * kRowScales, u = b_scale_unit<TJ>(wave);
    if (TI == 4 || wave < TI) dma16(p.sa, st.sa + 64 * wave * kRowScales, p.osa, os);
    if (TJ == 4 || u < TJ) dma16(p.sb, st.sb + 64 * u * kRowScales, p.osb, os);
  }
}
template <int TI, int TJ, bool kGate>
__device__ __forceinline__ void stage_load(LdsStage<TI, TJ>& st, const LdsOperands& p, int sc,
                                           int wave) {
#pragma unroll
  for (int j = 0; j < kLoadParts<TI, TJ>; ++j) stage_load_part<TI, TJ, kGate>(st, p, sc, wave, j);
}

template <bool kHi>
__device__ __forceinline__ h2 scale_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, kHi);
}

__device__ __forceinline__ uint4 lds_granule(const uint8_t* base, int row, int g) {
  return *reinterpret_cast<const uint4*>(base + row * kRowBytes + ((g ^ ((row >> 1) & 7)) << 4));
}

// E4M3 scale pairs of granule group gq as fp16 pairs (d[i][0] for the group's first 16
// k values, d[i][1] for the next 16).
template <int T>
__device__ __forceinline__ void group_scales(const uint2 (&sc)[T], int gq, h2 (&d)[T][2]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const uint32_t w = (gq < 2) ? sc[i].x : sc[i].y;
    const h2 pr = (gq & 1) ? scale_pair<true>(w) : scale_pair<false>(w);
    d[i][0] = h2{pr.x, pr.x};
    d[i][1] = h2{pr.y, pr.y};
  }
}

// Multiply one super-chunk held in LDS: 16 k-steps of TI TJ MFMAs (4 granule groups of
// 4 k-steps).  Software-pipelined: the operands of k-step s + 1 are dequantized while
// the MFMAs of k-step s issue (at 4 x 4 one MFMA, then up to five VALU instructions,
// repeated), so the conversion runs in the MFMA pipe's shadow instead of in front of
// it; the next group's granules are read from LDS three k-steps before they are used.
// With kLoad, the copies of super-chunk `next_sc` into `next` go out two per k-step
// in the first k-steps (0-8 at 4 x 4), right after the k-step's first MFMA, which leaves
// the others for them to land.  (Issued in one burst, they hold up the wave's in-order
// instruction stream while the matrix pipe idles.)
// With kTail, K ends `blocks` 16-value blocks into the super-chunk (a multiple of 4): what
// the copies bring behind it are other rows' values, and their scales are cleared.
template <int TI, int TJ, bool kLoad, bool kGate, bool kTail>
__device__ __forceinline__ void stage_mma(const LdsStage<TI, TJ>& st, f32x16 (&acc)[TI][TJ], int ra,
                                          int rb, int h, LdsStage<TI, TJ>& next,
                                          const LdsOperands& p, int next_sc, int wave, int blocks) {
  uint2 sca[TI], scb[TJ];
  uint4 ga[TI], gb[TJ], na[TI], nb[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    sca[i] = *reinterpret_cast<const uint2*>(st.sa + (ra + 32 * i) * kRowScales + 8 * h);
    ga[i] = lds_granule(st.a, ra + 32 * i, 4 * h);
  }
#pragma unroll
  for (int i = 0; i < TJ; ++i) {
    scb[i] = *reinterpret_cast<const uint2*>(st.sb + (rb + 32 * i) * kRowScales + 8 * h);
    gb[i] = lds_granule(st.b, rb + 32 * i, 4 * h);
  }
  if constexpr (kTail) {
    const bool first = blocks - 8 * h >= 4, last = blocks - 8 * h >= 8;
#pragma unroll
    for (int i = 0; i < TI; ++i) sca[i] = make_uint2(first ? sca[i].x : 0, last ? sca[i].y : 0);
#pragma unroll
    for (int i = 0; i < TJ; ++i) scb[i] = make_uint2(first ? scb[i].x : 0, last ? scb[i].y : 0);
  }
  h2 da[TI][2], db[TJ][2];
  group_scales(sca, 0, da);
  group_scales(scb, 0, db);
  h8 A[TI], B[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i) A[i] = dequant8(word(ga[i], 0), da[i][0]);
#pragma unroll
  for (int i = 0; i < TJ; ++i) B[i] = dequant8(word(gb[i], 0), db[i][0]);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    const int gq = s >> 2, jj = s & 3;
    if (jj == 0 && gq < 3) {
#pragma unroll
      for (int i = 0; i < TI; ++i) na[i] = lds_granule(st.a, ra + 32 * i, 4 * h + gq + 1);
#pragma unroll
      for (int i = 0; i < TJ; ++i) nb[i] = lds_granule(st.b, rb + 32 * i, 4 * h + gq + 1);
    }
    h8 An[TI], Bn[TJ];
    if (s < 15) {
      const int gq1 = (s + 1) >> 2, jj1 = (s + 1) & 3;
      if (jj1 == 0) {
#pragma unroll
        for (int i = 0; i < TI; ++i) ga[i] = na[i];
#pragma unroll
        for (int i = 0; i < TJ; ++i) gb[i] = nb[i];
        group_scales(sca, gq1, da);
        group_scales(scb, gq1, db);
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) An[i] = dequant8(word(ga[i], jj1), da[i][jj1 >> 1]);
#pragma unroll
      for (int i = 0; i < TJ; ++i) Bn[i] = dequant8(word(gb[i], jj1), db[i][jj1 >> 1]);
    }
    const bool copies = kLoad && s < kLoadParts<TI, TJ>;
    if (copies) stage_load_part<TI, TJ, kGate>(next, p, next_sc, wave, s);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int n = 0; n < TJ; ++n)
        acc[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[i], B[n], acc[i][n], 0, 0, 0);
    if (jj == 0 && gq < 3) __builtin_amdgcn_sched_group_barrier(0x100, TI + TJ, 0);  // LDS reads
    constexpr int kMfmas = TI * TJ, kValu = (10 * (TI + TJ) + kMfmas - 1) / kMfmas;
#pragma unroll
    for (int m = 0; m < kMfmas; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
      if (copies && m == 0) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);   // the copies
      __builtin_amdgcn_sched_group_barrier(0x002, kValu, 0);   // then up to five VALU at 4 x 4
    }
    __builtin_amdgcn_sched_barrier(0);
    if (s < 15) {
#pragma unroll
      for (int i = 0; i < TI; ++i) A[i] = An[i];
#pragma unroll
      for (int i = 0; i < TJ; ++i) B[i] = Bn[i];
    }
  }
}

// The products of super-chunks first, first + kSplit, .. (nsc of them), through two stages.
// Each step: wait for this wave's copies of the stage about to be used, barrier
// (so every wave's copies have landed and the other stage is no longer read), then
// multiply while copying the next super-chunk into the other stage.  A single-exit
// loop keeps the 256 accumulator registers in place.
// With `idle` (a wave whose rows or columns are all outside of Y) it copies only.
template <int TI, int TJ, int kSplit, bool kGate, bool kTail>
__device__ __forceinline__ void lds_products(LdsStage<TI, TJ>& st0, LdsStage<TI, TJ>& st1,
                                             const LdsOperands& p, f32x16 (&acc)[TI][TJ], int ra,
                                             int rb, int h, int wave, int first, int nsc,
                                             int blocks, bool idle) {
  auto chunk = [&](int i) { return kSplit * i + first; };
  // with a split the last of them may be past the end: any copy does, its scales are cleared
  auto copied = [&](int i) {
    return kSplit == 1 ? chunk(i) : min(chunk(i), (blocks - 1) / 16);
  };
  stage_load<TI, TJ, kGate>(st0, p, copied(0), wave);
  int i = 0;
  for (; i + 1 < nsc; i += 2) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (kSplit == 4 && idle) stage_load<TI, TJ, kGate>(st1, p, copied(i + 1), wave);
    else stage_mma<TI, TJ, true, kGate, false>(st0, acc, ra, rb, h, st1, p, copied(i + 1), wave, 16);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    // unconditional (a redundant copy of the last super-chunk when none is left): a
    // branch here lets the compiler sink the previous stage's MFMAs past the barrier
    if (kSplit == 4 && idle) stage_load<TI, TJ, kGate>(st0, p, copied(min(i + 2, nsc - 1)), wave);
    else
      stage_mma<TI, TJ, true, kGate, kTail>(st1, acc, ra, rb, h, st0, p, copied(min(i + 2, nsc - 1)),
                                            wave, blocks - 16 * chunk(i + 1));
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (i < nsc && !(kSplit == 4 && idle))
    stage_mma<TI, TJ, false, kGate, kTail>(st0, acc, ra, rb, h, st1, p, 0, wave,
                                           blocks - 16 * chunk(i));
}

constexpr int waves_per_simd(int mfma_tiles, int split) {
  return mfma_tiles == 16 ? 1 : split == 4 ? 4 : 2;
}

// Tile (64 TI) x (64 TJ), TI x TJ MFMA tiles to a wave.  4 x 4 fills a CU with one workgroup
// (LDS and registers); of 2 x 2 two run beside each other.  With a split, kSplit groups of four
// waves share one tile, each with every kSplit-th super-chunk: for so few tiles that a CU has
// no second one.
template <int TI, int TJ, int kEpi, bool kTail, int kSplit>
__global__ __attribute__((amdgpu_flat_work_group_size(256 * kSplit, 256 * kSplit),
                          amdgpu_waves_per_eu(waves_per_simd(TI * TJ, kSplit), waves_per_simd(TI * TJ, kSplit))))
void qlinear_lds_kernel(const uint8_t* __restrict__ xd, const uint8_t* __restrict__ xs,
                        const float* __restrict__ xt, const uint8_t* __restrict__ wd,
                        const uint8_t* __restrict__ ws, const float* __restrict__ wt, int M,
                        int N, int K, int tiles_m, int tiles_n, void* __restrict__ y,
                        EpilogueArgs e) {
  constexpr bool kGate = kEpi == kGated;
  constexpr int kProj = kGate ? 2 : 1;   // weight rows of one column of Y
  constexpr int kBM = 64 * TI, kBN = 64 * TJ;
  __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st0;
  __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st1;
  // ---- tile assignment: contiguous range per XCD, grouped along M inside it
  const TileCoord tc = tile_of(blockIdx.x, tiles_m, tiles_n);
  const int tm = tc.tm, tn = tc.tn;

  // the wave index is made explicitly uniform so that the LDS destinations of the
  // direct loads (M0) are scalar values rather than per-lane registers
  const int lane = threadIdx.x & 63;
  const int group = kSplit == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) - 4 * group;
  const int lr = lane & 31, h = lane >> 5;
  const uint32_t kb2 = K / 2, kb16 = K / 16;

  LdsOperands p;
  p.a = __builtin_amdgcn_make_buffer_rsrc((void*)xd, 0, (int)((uint32_t)M * kb2), kRsrcWord3);
  p.sa = __builtin_amdgcn_make_buffer_rsrc((void*)xs, 0, (int)((uint32_t)M * kb16), kRsrcWord3);
  p.b = __builtin_amdgcn_make_buffer_rsrc((void*)wd, 0, (int)((uint32_t)(kProj * N) * kb2), kRsrcWord3);
  p.sb = __builtin_amdgcn_make_buffer_rsrc((void*)ws, 0, (int)((uint32_t)(kProj * N) * kb16), kRsrcWord3);
  // the weight row behind row r of the tile
  auto weight_row = [&](int r) -> uint32_t {
    if constexpr (!kGate) return tn * kBN + r;
    bool up;
    const int g = gated_row(r, up);
    return tn * (kBN / 2) + g + (up ? N : 0);
  };
  {
    // DMA lane l of row-group q writes LDS slot (l & 7) of local row kBM/4*wave + 8*q +
    // (l >> 3); it fetches the granule that the swizzle puts in that slot:
    // g = slot ^ ((row >> 1) & 7) = slot ^ (((l >> 4) + 4 * (q & 1)) & 7).
    const int sub = lane >> 3, slot = lane & 7;
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const uint32_t g = slot ^ (((sub >> 1) + 4 * par) & 7);
      p.oa[par] = (uint32_t)(tm * kBM + 16 * TI * wave + sub) * kb2 + 16 * g;
      p.ob[par] = weight_row(16 * TJ * wave + sub) * kb2 + 16 * g;
      p.ou[par] = p.ob[par] + (uint32_t)N * kb2;
    }
    p.group_stride = 8 * kb2;
    p.osa = (uint32_t)(tm * kBM + 64 * wave + lane) * kb16;
    p.osb = weight_row(64 * b_scale_unit<TJ>(wave) + lane) * kb16;
  }

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int n = 0; n < TJ; ++n) acc[i][n] = f32x16{};

  // Where the wave is in the tile.  Of a tile in four groups the waves of the same place are
  // on different SIMDs: what the last rows and columns leave idle is the same for all of them
  // (16 x 4096 x 4096: 11.2 us, 14.7 where they multiply zeros).
  const int place = kSplit == 4 ? (wave + group) & 3 : wave;
  const int ra = (place >> 1) * (32 * TI) + lr;    // this lane's first A row in the tile
  const int rb = (place & 1) * (32 * TJ) + lr;     // and first B row
  const bool idle = tm * kBM + (place >> 1) * (32 * TI) >= M ||
                    (kGate ? tn * (kBN / 2) : tn * kBN + (place & 1) * (32 * TJ)) >= N;
  const int nsc = (K + kSuper * kSplit - 1) / (kSuper * kSplit), blocks = K / 16;
  if constexpr (kSplit == 1) {
    lds_products<TI, TJ, 1, kGate, kTail>(st0, st1, p, acc, ra, rb, h, wave, 0, nsc, blocks, idle);
  } else {
    __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st2;
    __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st3;
    // branches, not sets of pointers: the compiler has to know which stage a copy goes to, or
    // it waits for it before the next read
    if (group == 0)
      lds_products<TI, TJ, kSplit, kGate, true>(st0, st1, p, acc, ra, rb, h, wave, 0, nsc, blocks, idle);
    else if (group == 1)
      lds_products<TI, TJ, kSplit, kGate, true>(st2, st3, p, acc, ra, rb, h, wave, 1, nsc, blocks, idle);
    if constexpr (kSplit == 4) {
      __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st4;
      __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st5;
      __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st6;
      __shared__ __attribute__((aligned(16))) LdsStage<TI, TJ> st7;
      if (group == 2)
        lds_products<TI, TJ, 4, kGate, true>(st4, st5, p, acc, ra, rb, h, wave, 2, nsc, blocks, idle);
      else if (group == 3)
        lds_products<TI, TJ, 4, kGate, true>(st6, st7, p, acc, ra, rb, h, wave, 3, nsc, blocks, idle);
      static_assert(TI == 1 && TJ == 1 && kJoinBytes <= sizeof(LdsStage<TI, TJ>),
                    "the sums take the stages' place");
      store_joined<kGate>(e, y, M, N, tm, tn, wave, place, group, lane, xt[0] * wt[0], acc[0][0],
                          [&](int g, int half) {
                            return (g == 0 ? st0 : g == 1 ? st2 : g == 2 ? st4 : st6).a + half * kJoinBytes / 2;
                          });
      return;
    } else {
      // each group gets the other's sums of half of the wave's rows, and finishes those
      static_assert(TI == 2 && TJ * 256 * sizeof(f32x16) <= sizeof(LdsStage<TI, TJ>),
                    "the sums take the stages' place");
      const int at = 64 * wave + lane;
      f32x16 half[1][TJ];
      auto give = [&](LdsStage<TI, TJ>& to, int i) {
#pragma unroll
        for (int n = 0; n < TJ; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            reinterpret_cast<f32x4*>(to.a)[(4 * n + q) * 256 + at] =
                f32x4{acc[i][n][4 * q], acc[i][n][4 * q + 1], acc[i][n][4 * q + 2], acc[i][n][4 * q + 3]};
      };
      auto take = [&](const LdsStage<TI, TJ>& from, int i) {
#pragma unroll
        for (int n = 0; n < TJ; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = reinterpret_cast<const f32x4*>(from.a)[(4 * n + q) * 256 + at];
#pragma unroll
            for (int k = 0; k < 4; ++k) half[0][n][4 * q + k] = acc[i][n][4 * q + k] + v[k];
          }
      };
      __syncthreads();   // every wave has read its operands
      if (group == 0) give(st0, 1);
      else give(st1, 0);
      __syncthreads();
      if (group == 0) take(st1, 0);
      else take(st0, 1);
      store_fused<1, TJ, kGate>(e, y, M, N, tm * kBM + (wave >> 1) * (32 * TI) + 32 * group,
                                (tn * kBN + (wave & 1) * (32 * TJ)) / kProj, lane, xt[0] * wt[0], half);
      return;
    }
  }

  if constexpr (kEpi == kPlain) {
    static_assert(TI == 4 && TJ == 4, "the plain store takes a whole tile");
    store_tile(static_cast<uint16_t*>(y), M, N, tm, tn, wave, lr, h, xt[0] * wt[0], acc);
  } else if constexpr (kSplit == 1) {
    store_fused<TI, TJ, kGate>(e, y, M, N, tm * kBM + (wave >> 1) * (32 * TI),
                               (tn * kBN + (wave & 1) * (32 * TJ)) / kProj, lane_again(), xt[0] * wt[0], acc);
  }
}

template <int TI, int TJ, int kEpi, int kSplit = 1>
hipError_t launch_lds(const uint8_t* xd, const uint8_t* xs, const float* xt, const uint8_t* wd,
                      const uint8_t* ws, const float* wt, int64_t M, int64_t N, int64_t K,
                      void* y, const EpilogueArgs& e, hipStream_t s) {
  constexpr int kCols = 64 * TJ / (kEpi == kGated ? 2 : 1), kThreads = 256 * kSplit;
  const int tiles_m = (int)((M + 64 * TI - 1) / (64 * TI));
  const int tiles_n = (int)((N + kCols - 1) / kCols);
  if constexpr (kEpi == kPlain || kSplit > 1)   // a split clears what is behind K anyway
    qlinear_lds_kernel<TI, TJ, kEpi, false, kSplit><<<tiles_m * tiles_n, kThreads, 0, s>>>(
        xd, xs, xt, wd, ws, wt, (int)M, (int)N, (int)K, tiles_m, tiles_n, y, e);
  else if (K % kSuper == 0)
    qlinear_lds_kernel<TI, TJ, kEpi, false, 1><<<tiles_m * tiles_n, kThreads, 0, s>>>(
        xd, xs, xt, wd, ws, wt, (int)M, (int)N, (int)K, tiles_m, tiles_n, y, e);
  else
    qlinear_lds_kernel<TI, TJ, kEpi, true, 1><<<tiles_m * tiles_n, kThreads, 0, s>>>(
        xd, xs, xt, wd, ws, wt, (int)M, (int)N, (int)K, tiles_m, tiles_n, y, e);
  return hipGetLastError();
}

template <int TI, int TJ, int STAGES, int WPE>
hipError_t launch_cfg(const uint8_t* xd, const uint8_t* xs, const float* xt, const uint8_t* wd,
                      const uint8_t* ws, const float* wt, int64_t M, int64_t N, int64_t K,
                      uint16_t* y, hipStream_t s) {
  constexpr int kBM = 64 * TI, kBN = 64 * TJ;
  const int tiles_m = (int)((M + kBM - 1) / kBM);
  const int tiles_n = (int)((N + kBN - 1) / kBN);
  qlinear_kernel<TI, TJ, STAGES, WPE><<<tiles_m * tiles_n, 256, 0, s>>>(
      xd, xs, xt, wd, ws, wt, (int)M, (int)N, (int)K, tiles_m, tiles_n, y);
  return hipGetLastError();
}

// Tile of an epilogue's product, by what a round of workgroups takes (us, measured with silu:
// fixed, and per 4096 of K): 64 x 64 with K split over four groups of waves, while every tile
// has a CU of its own; 128 x 128, two workgroups to a CU or one (half a round, or all
// that there is: then of eight waves that split K); 256 x 256, which converts a value for
// twice as many products, where it fills the GPU.  In this order: 16 x 4096 x 4096 11.2, 29.0,
// 31.5 and 77 us; 256 x 4096 x 4096 16.9, 29.7, 31.9 and 77; 64 x 4096 x 512 7.5, 8.4, 8.9 and
// 23; 333 x 8198 x 4160 -, 39, 40 and 90; 2048 x 4096 x 4096 -, 69, 65 and 90; 4096 x 4096 x
// 4096 -, -, 125 and 110.  (All measured with an earlier epilogue; the chosen ones now take 10.5,
// 16, 9.0 from Python, 34, 61 and 101.)
struct QShape {
  int t, split, resident;
  float half, half_k, full, full_k;
};
constexpr QShape kQShapes[] = {{1, 4, 256, 5.0f, 9.5f, 6.0f, 10.5f},
                               {2, 2, 256, 4.5f, 27.0f, 4.5f, 27.0f},
                               {2, 1, 512, 4.0f, 33.0f, 3.0f, 60.0f},
                               {4, 1, 256, 15.5f, 84.0f, 15.5f, 84.0f}};
int64_t tiles_of(const QLinearArgs& a, const QShape& h) {
  const int64_t rows = 64 * h.t, cols = a.gated ? rows / 2 : rows;
  return ((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols);
}
const QShape& shape_of(const QLinearArgs& a) {
  const QShape* best = nullptr;
  float least = 0.0f;
  const float k = (float)a.K / 4096.0f;
  for (const QShape& h : kQShapes) {
    const int64_t tiles = tiles_of(a, h), full = tiles / h.resident, rest = tiles % h.resident;
    // no second super-chunk to split, or more than one round
    if (h.split > 1 && (a.K <= kSuper || tiles > h.resident)) continue;
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
hipError_t launch_epi(const QLinearArgs& a, hipStream_t s) {
  const QShape& h = shape_of(a);
  const auto launch = h.split == 4   ? launch_lds<1, 1, kEpi, 4>
                      : h.split == 2 ? launch_lds<2, 2, kEpi, 2>
                      : h.t == 2     ? launch_lds<2, 2, kEpi>
                                     : launch_lds<4, 4, kEpi>;
  return launch(a.xd, a.xs, a.xt, a.wd, a.ws, a.wt, a.M, a.N, a.K, a.y, a.e, s);
}

}  // namespace

// Both kernels tile the output in 256 x 256 blocks (launch_cfg<4, 4, ...>: 64 * 4).
int64_t qlinear_grid(int64_t M, int64_t N) {
  static_assert(64 * 4 == kTileRows, "both qlinear kernels use the same output tile");
  return ((M + kTileRows - 1) / kTileRows) * ((N + kTileRows - 1) / kTileRows);
}

hipError_t launch_qlinear(const uint8_t* xd, const uint8_t* xs, const float* xt,
                          const uint8_t* wd, const uint8_t* ws, const float* wt, int64_t M,
                          int64_t N, int64_t K, uint16_t* y, hipStream_t s) {
  // K in whole 256-wide super-chunks: LDS-staged kernel; otherwise (K % 64 == 0) the
  // register-staged kernel
  if (K % kSuper == 0)
    return launch_lds<4, 4, kPlain>(xd, xs, xt, wd, ws, wt, M, N, K, y, EpilogueArgs{}, s);
  return launch_cfg<4, 4, 3, 1>(xd, xs, xt, wd, ws, wt, M, N, K, y, s);
}

int64_t qlinear_epilogue_grid(const QLinearArgs& a) { return tiles_of(a, shape_of(a)); }

hipError_t launch_qlinear_epilogue(const QLinearArgs& a, hipStream_t s) {
  return a.gated ? launch_epi<kGated>(a, s) : launch_epi<kFused>(a, s);
}

}  // namespace fos
