// Epilogue of the GEMM kernels' tiles with bias, activation, gate and residual, from the
// accumulators' own layout: element a of lane (lr, h) is row (a & 3) + 8 (a >> 2) + 4h and
// column lr of a 32x32 tile.  Nothing of it overlaps the products of its own workgroup, and
// its arithmetic bounds it: a wave alone on its SIMD (the 256x256 tile, 256 values a lane)
// issues a VALU instruction every 8 cycles.  8192 x 12288 x 4096 NVFP4, six rounds of tiles:
// 581 us without an activation, 606 with silu, 659 with gelu, 611 with Z kept, 646 with a
// residual, beside 576 for the plain product.  (Eight waves of 128 x 64, two to a SIMD, take
// less for the epilogue and convert each operand more often: 645, 655, 682 and 719 without a
// residual.)
#pragma once

#include "activation.hpp"
#include "gemm_common.hpp"

namespace fos {
namespace gemm {

// What a GEMM kernel does with its sums: kPlain stores them, kFused applies the epilogue,
// kGated too, with gate and other projection in neighbouring 32-column tiles.
enum { kPlain, kFused, kGated };

// Weight row behind row r (0 .. 64 TJ - 1) of a gated tile, without the tile's first column:
// rows come in groups of 32, gate and other projection in turn; `up` says which.
__device__ __forceinline__ int gated_row(int r, bool& up) {
  up = (r >> 5) & 1;
  return ((r >> 6) << 5) | (r & 31);
}

// A wave's rows of a row-major matrix as a buffer resource: what lies outside of it is not
// stored and reads as zero, which takes care of the last rows.  A column outside gets an
// offset outside (kNowhere); with at most kMaxEpilogueCols columns and kMaxResidualStride
// (the host checks) 128 rows end below it.
constexpr uint32_t kNowhere = 0x80000000u;
struct RowWindow {
  __amdgpu_buffer_rsrc_t r;
  uint32_t row_bytes;
};
__device__ __forceinline__ RowWindow row_window(const void* p, int64_t first, int rows,
                                                int64_t stride, int cols, int bytes) {
  RowWindow w;
  w.row_bytes = (uint32_t)stride * bytes;
  w.r = __builtin_amdgcn_make_buffer_rsrc(
      (char*)p + first * stride * bytes, 0,
      rows > 0 ? (int)((rows - 1) * w.row_bytes + (uint32_t)cols * bytes) : 0, kRsrcWord3);
  return w;
}

// Adjacent lanes swap halves of a packed pair: from (row r, row r + 1) of the lane's own
// column to the even lane's row r, columns (c, c + 1) and the odd lane's row r + 1, columns
// (c - 1, c), and (unswap) back.
__device__ __forceinline__ uint32_t swap_pairs(uint32_t p, int odd) {
  const uint32_t q = __builtin_amdgcn_update_dpp(0u, p, 0xB1, 0xF, 0xF, false);
  return __builtin_amdgcn_perm(q, p, odd ? 0x03020706u : 0x05040100u);
}

// The 16 values of one 32x32 tile of bf16 in packed pairs of rows (a, a + 1): stored, or
// loaded.  `row`: the tile's first row in the window; `col`: the lane's column, kNowhere if
// there is none.  kPair: 4-byte accesses of two columns (even columns, 4-byte alignment).
template <bool kPair>
__device__ __forceinline__ uint32_t tile_offset(const RowWindow& w, int row, uint32_t col, int h, int odd) {
  if (col == kNowhere) return col;
  return kPair ? (row + 4 * h + odd) * w.row_bytes + 2 * (col - odd) : (row + 4 * h) * w.row_bytes + 2 * col;
}
__device__ __forceinline__ int tile_row_offset(const RowWindow& w, int a) {
  return (int)(((a & 3) + 8 * (a >> 2)) * w.row_bytes);
}
__device__ __forceinline__ void store_bf16_tile(const RowWindow& w, const uint32_t (&v)[8], int row,
                                                uint32_t col, int h, int odd, bool pair) {
  if (pair) {
    const uint32_t at = tile_offset<true>(w, row, col, h, odd);
#pragma unroll
    for (int a = 0; a < 16; a += 2)
      __builtin_amdgcn_raw_buffer_store_b32(swap_pairs(v[a / 2], odd), w.r, at, tile_row_offset(w, a), 0);
  } else {
    const uint32_t at = tile_offset<false>(w, row, col, h, odd);
#pragma unroll
    for (int a = 0; a < 16; ++a)
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[a / 2] >> (16 * (a & 1))), w.r, at,
                                            tile_row_offset(w, a), 0);
  }
}
// As they are in memory: kPair 8 words of two columns each, else 16 values.
template <bool kPair>
__device__ __forceinline__ void load_bf16_tile(const RowWindow& w, uint32_t (&v)[kPair ? 8 : 16], int row,
                                               uint32_t col, int h, int odd) {
  const uint32_t at = tile_offset<kPair>(w, row, col, h, odd);
#pragma unroll
  for (int a = 0; a < 16; a += kPair ? 2 : 1) {
    if constexpr (kPair) v[a / 2] = __builtin_amdgcn_raw_buffer_load_b32(w.r, at, tile_row_offset(w, a), 0);
    else v[a] = __builtin_amdgcn_raw_buffer_load_b16(w.r, at, tile_row_offset(w, a), 0);
  }
}

// The lane, asked for again where the register that held it is worth more in the loop before.
__device__ __forceinline__ int lane_again() {
  return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
}

// The tile of a wave, rows m0 .. and columns n0 .. of y: act(s acc + bias) (times the other
// projection) + residual.  A tile's residual is on its way while the tile before is computed, with
// single columns while the tile itself is.  Without a residual nothing of it is in the loop (asked
// for tile by tile, it took 27 us more without an activation).
template <int TI, int TJ, bool kGate, bool kRes, int kAct>
__device__ __forceinline__ void store_fused_as(const EpilogueArgs& e, void* y, int M, int N, int m0,
                                               int n0, int lane, float s,
                                               const f32x16 (&acc)[TI][TJ]) {
  constexpr int kStep = kGate ? 2 : 1, kTiles = TJ / kStep;
  const int lr = lane & 31, h = lane >> 5, odd = lr & 1;
  const int rows = min(32 * TI, M - m0);
  const bool pair = e.pair;
  const RowWindow wy = row_window(y, m0, rows, N, N, e.f32_out ? 4 : 2);
  const RowWindow wz = row_window(e.preact, m0, e.preact ? rows : 0, kStep * (int64_t)N, kStep * N, 2);
  const RowWindow wr = row_window(e.residual, m0, kRes ? rows : 0, e.residual_stride, N, 2);
  uint32_t col[kTiles];
  float bias[kTiles], bias_up[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int n = n0 + 32 * t + lr;
    col[t] = n < N ? (uint32_t)n : kNowhere;
    bias[t] = bias_up[t] = 0.0f;
    if (e.bias && n < N) {
      bias[t] = bf16_lo(e.bias[n]);
      if (kGate) bias_up[t] = bf16_lo(e.bias[N + n]);
    }
  }
  // (arrays of their own: one that holds either layout is kept in scratch memory)
  uint32_t next[8] = {};
  if (kRes && pair) load_bf16_tile<true>(wr, next, 0, col[0], h, odd);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      uint32_t res[8], one[16];
#pragma unroll
      for (int a = 0; a < 8; ++a) res[a] = next[a];
      if (kRes) {
        if (!pair)
          load_bf16_tile<false>(wr, one, 32 * i, col[t], h, odd);
        else if (i + 1 < TI || t + 1 < kTiles)
          load_bf16_tile<true>(wr, next, 32 * (t + 1 < kTiles ? i : i + 1), col[(t + 1) % kTiles], h, odd);
      }
      float v[16];
      uint32_t z[8], zu[8];
#pragma unroll
      for (int a = 0; a < 16; a += 2) {
        float g[2], u[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          g[b] = __builtin_fmaf(acc[i][kStep * t][a + b], s, bias[t]);
          v[a + b] = activate<kAct>(g[b]);
          if constexpr (kGate) {
            u[b] = __builtin_fmaf(acc[i][kStep * t + 1][a + b], s, bias_up[t]);
            v[a + b] *= u[b];
          }
        }
        z[a / 2] = pack_bf16x2(g[0], g[1]);
        if constexpr (kGate) zu[a / 2] = pack_bf16x2(u[0], u[1]);
      }
      if (e.preact) {
        store_bf16_tile(wz, z, 32 * i, col[t], h, odd, pair);
        if constexpr (kGate)
          store_bf16_tile(wz, zu, 32 * i, col[t] == kNowhere ? kNowhere : col[t] + N, h, odd, pair);
      }
      if (kRes && pair) {
#pragma unroll
        for (int a = 0; a < 16; a += 2) {
          const uint32_t r = swap_pairs(res[a / 2], odd);
          v[a] += bf16_lo(r);
          v[a + 1] += bf16_hi(r);
        }
      } else if (kRes) {
#pragma unroll
        for (int a = 0; a < 16; ++a) v[a] += bf16_lo(one[a]);
      }
      if (e.f32_out) {
        const uint32_t at = col[t] == kNowhere ? kNowhere : (32 * i + 4 * h) * wy.row_bytes + 4 * col[t];
#pragma unroll
        for (int a = 0; a < 16; ++a)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[a]), wy.r, at,
                                                (int)(((a & 3) + 8 * (a >> 2)) * wy.row_bytes), 0);
      } else {
#pragma unroll
        for (int a = 0; a < 16; a += 2) z[a / 2] = pack_bf16x2(v[a], v[a + 1]);
        store_bf16_tile(wy, z, 32 * i, col[t], h, odd, pair);
      }
    }
  }
}

template <int TI, int TJ, bool kGate, bool kRes>
__device__ __forceinline__ void store_fused_act(const EpilogueArgs& e, void* y, int M, int N, int m0, int n0,
                                                int lane, float s, const f32x16 (&acc)[TI][TJ]) {
  switch (e.act) {
    case kActRelu: store_fused_as<TI, TJ, kGate, kRes, kActRelu>(e, y, M, N, m0, n0, lane, s, acc); break;
    case kActGelu: store_fused_as<TI, TJ, kGate, kRes, kActGelu>(e, y, M, N, m0, n0, lane, s, acc); break;
    case kActGeluTanh: store_fused_as<TI, TJ, kGate, kRes, kActGeluTanh>(e, y, M, N, m0, n0, lane, s, acc); break;
    case kActSilu: store_fused_as<TI, TJ, kGate, kRes, kActSilu>(e, y, M, N, m0, n0, lane, s, acc); break;
    default: store_fused_as<TI, TJ, kGate, kRes, kActNone>(e, y, M, N, m0, n0, lane, s, acc);
  }
}
template <int TI, int TJ, bool kGate>
__device__ __forceinline__ void store_fused(const EpilogueArgs& e, void* y, int M, int N, int m0,
                                            int n0, int lane, float s, const f32x16 (&acc)[TI][TJ]) {
  if constexpr (!kGate) {   // with a gate there is no residual
    if (e.residual) return store_fused_act<TI, TJ, kGate, true>(e, y, M, N, m0, n0, lane, s, acc);
  }
  store_fused_act<TI, TJ, kGate, false>(e, y, M, N, m0, n0, lane, s, acc);
}

// The epilogue of a 64 x 64 tile whose K is split over four groups of four waves, each wave
// with one 32x32 tile of its group's sums (2 x 2, `at` counts them).  place(g, half): 16-byte
// aligned LDS for half of the kJoinBytes of group g's, which may hold operands that a wave
// still reads.  A wave of the first group sums a tile of Y in the groups' order (with a gate:
// waves 0 and 1, both projections, whose sums are two neighbouring waves').
constexpr int kJoinBytes = 256 * sizeof(f32x16);
template <bool kGate, typename Place>
__device__ __forceinline__ void store_joined(const EpilogueArgs& e, void* y, int M, int N, int tm,
                                             int tn, int wave, int at, int group, int lane,
                                             float s, const f32x16& acc, Place place) {
  constexpr int kProj = kGate ? 2 : 1;
  auto quarter = [&](int g, int q) {   // values 4q .. 4q + 3 of every lane
    return reinterpret_cast<f32x4*>(place(g, q >> 1)) + 256 * (q & 1);
  };
  __syncthreads();   // every wave has read its operands
#pragma unroll
  for (int q = 0; q < 4; ++q)
    quarter(group, q)[64 * at + lane] = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  if (group != 0 || wave >= 4 / kProj) return;
  f32x16 sum[1][kProj];
#pragma unroll
  for (int t = 0; t < kProj; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int l = 64 * (kProj * wave + t) + lane;
      f32x4 v = quarter(0, q)[l];
#pragma unroll
      for (int g = 1; g < 4; ++g) v += quarter(g, q)[l];
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[0][t][4 * q + k] = v[k];
    }
  store_fused<1, kProj, kGate>(e, y, M, N, 64 * tm + 32 * (kGate ? wave : wave >> 1),
                               kGate ? 32 * tn : 64 * tn + 32 * (wave & 1), lane, s, sum);
}

}  // namespace gemm
}  // namespace fos
