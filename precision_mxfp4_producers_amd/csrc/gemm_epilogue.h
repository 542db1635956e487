// Epilogue of the fast main loop's 256 x 256 tile: bias, activation, residual,
// bf16 or fp32 output.
#pragma once

#include "activation.h"
#include "gemm_core.h"

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

// The tile leaves through a private LDS slice per wave, as the plain product's
// does: 32 rows x 64 columns at a time (a 272-byte pitch: eight rows at one
// column land on distinct banks), read back sixteen lanes a row, so that a bf16
// row of the wave is one whole 128-byte line.
constexpr int kEPitch = 272;
constexpr int kESlice = 32 * kEPitch;
static_assert(8 * kESlice <= kSmemBytes, "the slices fit in the stage buffers");

// Rows m0 .. M - 1 and columns n0 .. N - 1 of the tile (N a multiple of 32).
__device__ __forceinline__ void store_epilogue(uint8_t* smem, const v16f (&acc)[4][2], const Epilogue& e, int64_t M,
                                               int64_t N, int64_t m0, int64_t n0, int wave, int lane, int wm, int wn,
                                               int hl) {
  uint8_t* const buf = smem + wave * kESlice;
  const int r = lane & 31, rr0 = lane >> 4, ch = lane & 15;
  const int64_t col = n0 + wn * 64 + 4 * ch;
  const bool in = col < N;
  float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (e.bias && in) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = e.bias_f32 ? static_cast<const float*>(e.bias)[col + u]
                        : bf16_bits_to_f32(static_cast<const uint16_t*>(e.bias)[col + u]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row0 = m0 + wm * 128 + 32 * i + rr0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(buf + r * kEPitch + (32 * j + 8 * g + 4 * hl) * 4) =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
    // other lanes' values are read below: the hardware keeps a wave's LDS
    // accesses in order, and this the compiler
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    float v[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 q = *reinterpret_cast<const float4*>(buf + (4 * k + rr0) * kEPitch + ch * 16);
      v[k][0] = q.x; v[k][1] = q.y; v[k][2] = q.z; v[k][3] = q.w;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if (e.bias) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u) v[k][u] = __fadd_rn(v[k][u], b[u]);
    }
    if (e.z) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (in && row0 + 4 * k < M)
          *reinterpret_cast<uint2*>(e.z + (row0 + 4 * k) * N + col) =
              make_uint2(bf16_pack2_rne(v[k][0], v[k][1]), bf16_pack2_rne(v[k][2], v[k][3]));
    }
    if (e.act != FP4_ACT_NONE)
      with_act(e.act, [&](auto act) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int u = 0; u < 4; ++u) v[k][u] = act_value<act()>(v[k][u]);
      });
    if (e.residual) {
      uint2 q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        q[k] = in && row0 + 4 * k < M ? *reinterpret_cast<const uint2*>(e.residual + (row0 + 4 * k) * e.ldr + col) : make_uint2(0u, 0u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k][0] = __fadd_rn(v[k][0], __uint_as_float(q[k].x << 16));
        v[k][1] = __fadd_rn(v[k][1], __uint_as_float(q[k].x & 0xFFFF0000u));
        v[k][2] = __fadd_rn(v[k][2], __uint_as_float(q[k].y << 16));
        v[k][3] = __fadd_rn(v[k][3], __uint_as_float(q[k].y & 0xFFFF0000u));
      }
    }
    if (e.y_f32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!in || row0 + 4 * k >= M) continue;
        v4f* const p = reinterpret_cast<v4f*>(static_cast<float*>(e.y) + (row0 + 4 * k) * e.ldy + col);
        v4f o = {v[k][0], v[k][1], v[k][2], v[k][3]};
        if (e.accumulate) {
          const v4f prev = *p;
#pragma unroll
          for (int u = 0; u < 4; ++u) o[u] = __fadd_rn(prev[u], o[u]);
        }
        if (e.stream) __builtin_nontemporal_store(o, p);
        else *p = o;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!in || row0 + 4 * k >= M) continue;
        typedef uint32_t v2u __attribute__((ext_vector_type(2)));
        v2u* const p = reinterpret_cast<v2u*>(static_cast<uint16_t*>(e.y) + (row0 + 4 * k) * e.ldy + col);
        const v2u o = {bf16_pack2_rne(v[k][0], v[k][1]), bf16_pack2_rne(v[k][2], v[k][3])};
        if (e.stream) __builtin_nontemporal_store(o, p);
        else *p = o;
      }
    }
  }
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

// An output that cannot stay in the 256 MB Infinity Cache for its reader goes
// past it (the plain product's rule).
inline bool streams(int64_t bytes) { return bytes > ((int64_t)192 << 20); }

// Number of bm x bn tiles, or -1 when it exceeds a grid's 2^31 - 1 workgroups.
inline int64_t tiles_of(int64_t m, int64_t bm, int64_t n, int64_t bn) {
  const int64_t tm = (m - 1) / bm + 1, tn = (n - 1) / bn + 1;
  if (m == 0 || n == 0) return 0;
  return tm > 0x7FFFFFFF / tn ? -1 : tm * tn;
}

}  // namespace mx
