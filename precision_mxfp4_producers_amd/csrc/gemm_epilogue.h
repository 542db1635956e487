// Epilogue of the fast main loop's 256 x 256 tile: bias, activation, residual,
// bf16 or fp32 output.
#pragma once

#include "activation.h"
#include "gemm_core.h"
#include "rows.h"

namespace mx {

// z = acc + bias, y = act(z) + residual, or y += acc.
struct Epilogue {
  void* y;                                               // [rows][ldy] bf16 or fp32
  int64_t ldy;
  const void* bias;                                      // [n] bf16 or fp32, or null
  const uint16_t* residual;                              // [rows][ldr] bf16, or null
  int64_t ldr;
  uint16_t* z;                                           // [rows][n] bf16, or null
  int act;
  int y_f32, bias_f32;
  int accumulate;                                        // fp32 y, nothing else
  int stream;                                            // y past the caches (non-temporal stores)
};

// Four or eight neighbouring values as bf16.
template <int W>
__device__ __forceinline__ void put_row(uint16_t* p, const float (&v)[W], int stream) {
  typedef uint32_t words __attribute__((ext_vector_type(W / 2)));
  words o;
#pragma unroll
  for (int u = 0; u < W / 2; ++u) {
    const bf16x2_t b = {(__bf16)v[2 * u], (__bf16)v[2 * u + 1]};   // a NaN stays one
    o[u] = __builtin_bit_cast(uint32_t, b);
  }
  put(reinterpret_cast<words*>(p), o, stream);
}

// The tile leaves through a private LDS slice per wave, as the plain product's
// does, 32 rows at a time, and is read back eight lanes a row, so that every
// store instruction writes eight whole 128-byte lines: a bf16 row of the wave is
// its 64 columns, eight a lane (16 bytes); an fp32 one 32 of them, four a lane,
// in two passes.  (Sixteen lanes a row and four rows an instruction, 256 bytes a
// row in fp32, is partly written lines.)
// Pitches of an odd number of 16-byte chunks keep 16 lanes on distinct banks.
//
// Whatever the epilogue reads is read, and waited for, before the first store:
// loads and stores leave one counter, and a wait for a load behind a store waits
// for the store too, which cost the products above another quarter.  PLAIN: no
// bias, activation, residual or z.
template <bool F32>
struct EpilogueTile {
  static constexpr int kPitch = F32 ? 144 : 272, kSlice = 32 * kPitch;
  static constexpr int kCols = F32 ? 32 : 64, kPer = F32 ? 4 : 8;
  static_assert(8 * kSlice <= kSmemBytes, "the slices fit in the stage buffers");
};

// Rows m0 .. M - 1 and columns n0 .. N - 1 of the tile (N a multiple of 32).
template <bool F32, bool PLAIN>
__device__ __forceinline__ void store_epilogue_as(uint8_t* smem, const v16f (&acc)[4][2], const Epilogue& e, int64_t M,
                                                  int64_t N, int64_t m0, int64_t n0, int wave, int lane, int wm, int wn,
                                                  int hl) {
  using T = EpilogueTile<F32>;
  constexpr int W = T::kPer, PASSES = 64 / T::kCols;
  uint8_t* const buf = smem + wave * T::kSlice;
  const int r = lane & 31, rr0 = lane >> 3, ch = lane & 7;
  // sub-tiles past the last row or column: a small product's last tile
  const int live_rows = (int)min(M - (m0 + wm * 128), (int64_t)128);
  if (live_rows <= 0 || n0 + wn * 64 >= N) return;
  float b[PASSES][W];
  uint32_t res[4][PASSES][4][W / 2];
  if constexpr (!PLAIN) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int64_t col = n0 + wn * 64 + p * T::kCols + W * ch;
#pragma unroll
      for (int u = 0; u < W; ++u) b[p][u] = 0.0f;
      if (e.bias && col < N) {
#pragma unroll
        for (int u = 0; u < W; ++u)
          b[p][u] = e.bias_f32 ? static_cast<const float*>(e.bias)[col + u]
                               : bf16_bits_to_f32(static_cast<const uint16_t*>(e.bias)[col + u]);
      }
      if (e.residual) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t row = m0 + wm * 128 + 32 * i + rr0 + 8 * k;
            const uint16_t* const q = e.residual + row * e.ldr + col;
            if constexpr (F32) {
              const uint2 v = col < N && row < M ? *reinterpret_cast<const uint2*>(q) : make_uint2(0u, 0u);
              res[i][p][k][0] = v.x; res[i][p][k][1] = v.y;
            } else {
              const uint4 v = col < N && row < M ? *reinterpret_cast<const uint4*>(q) : make_uint4(0u, 0u, 0u, 0u);
              res[i][p][k][0] = v.x; res[i][p][k][1] = v.y; res[i][p][k][2] = v.z; res[i][p][k][3] = v.w;
            }
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < W / 2; ++u) asm volatile("" : "+v"(res[i][p][k][u]));
      }
#pragma unroll
      for (int u = 0; u < W; ++u) asm volatile("" : "+v"(b[p][u]));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (32 * i >= live_rows) break;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int64_t row0 = m0 + wm * 128 + 32 * i + rr0, col = n0 + wn * 64 + p * T::kCols + W * ch;
      const bool in = col < N;
#pragma unroll
      for (int j = F32 ? p : 0; j < (F32 ? p + 1 : 2); ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(buf + r * T::kPitch + ((F32 ? 0 : 32 * j) + 8 * g + 4 * hl) * 4) =
              make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
      // other lanes' values are read below: the hardware keeps a wave's LDS
      // accesses in order, and this the compiler
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      float v[4][W];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < W / 4; ++q) {
          const float4 f = *reinterpret_cast<const float4*>(buf + (8 * k + rr0) * T::kPitch + (ch * W + 4 * q) * 4);
          v[k][4 * q] = f.x; v[k][4 * q + 1] = f.y; v[k][4 * q + 2] = f.z; v[k][4 * q + 3] = f.w;
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      if (!PLAIN && e.bias) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < W; ++u) v[k][u] = __fadd_rn(v[k][u], b[p][u]);
      }
      if (!PLAIN && e.z) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (in && row0 + 8 * k < M) put_row(e.z + (row0 + 8 * k) * N + col, v[k], e.stream);
      }
      if (!PLAIN && e.act != FP4_ACT_NONE)
        with_act(e.act, [&](auto act) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < W; ++u) v[k][u] = act_value<act(), F32>(v[k][u]);
        });
      if (!PLAIN && e.residual) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int u = 0; u < W; u += 2) {
            v[k][u] = __fadd_rn(v[k][u], __uint_as_float(res[i][p][k][u / 2] << 16));
            v[k][u + 1] = __fadd_rn(v[k][u + 1], __uint_as_float(res[i][p][k][u / 2] & 0xFFFF0000u));
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!in || row0 + 8 * k >= M) continue;
        if constexpr (F32) {
          v4f* const q = reinterpret_cast<v4f*>(static_cast<float*>(e.y) + (row0 + 8 * k) * e.ldy + col);
          v4f o = {v[k][0], v[k][1], v[k][2], v[k][3]};
          if (e.accumulate) {
            const v4f prev = *q;
#pragma unroll
            for (int u = 0; u < 4; ++u) o[u] = __fadd_rn(prev[u], o[u]);
          }
          put(q, o, e.stream);
        } else {
          put_row(static_cast<uint16_t*>(e.y) + (row0 + 8 * k) * e.ldy + col, v[k], e.stream);
        }
      }
    }
  }
}

template <bool PLAIN>
__device__ __forceinline__ void store_epilogue(uint8_t* smem, const v16f (&acc)[4][2], const Epilogue& e, int64_t M,
                                               int64_t N, int64_t m0, int64_t n0, int wave, int lane, int wm, int wn,
                                               int hl) {
  if (e.y_f32) store_epilogue_as<true, PLAIN>(smem, acc, e, M, N, m0, n0, wave, lane, wm, wn, hl);
  else store_epilogue_as<false, PLAIN>(smem, acc, e, M, N, m0, n0, wave, lane, wm, wn, hl);
}

__device__ __forceinline__ void zero_tile(v16f (&acc)[4][2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
}

// Row lengths by the main loop's K range (see kWindow).
inline int k_mode(int64_t k) { return k > 0 && k % 256 == 0 ? kWhole : (k >= 256 ? kWindow : kShort); }

// Most tiles of a launch.
constexpr int64_t kMostTiles = 0x7FFF0000;

// Number of bm x bn tiles, or -1 past kMostTiles.
inline int64_t tiles_of(int64_t m, int64_t bm, int64_t n, int64_t bn) {
  const int64_t tm = (m - 1) / bm + 1, tn = (n - 1) / bn + 1;
  if (m == 0 || n == 0) return 0;
  return tm > kMostTiles / tn ? -1 : tm * tn;
}

// Workgroups of so many tiles, one each.  A launch's dimension holds less than 2^32
// threads (a larger one wraps, with no error), which workgroups of 512 reach at 2^23
// tiles: past half of that they go to a second dimension, in equal shares of whole
// eights (one for each XCD).  The few spare ones come last.
constexpr int64_t kGridTiles = 1 << 22;
inline dim3 tile_grid(int64_t tiles) {
  const int64_t y = (tiles + kGridTiles - 1) / kGridTiles;
  return y > 1 ? dim3((unsigned)(((tiles + y - 1) / y + 7) / 8 * 8), (unsigned)y) : dim3((unsigned)tiles);
}
__device__ __forceinline__ int64_t grid_tile() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace mx
