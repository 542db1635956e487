// Block-scaled E2M1 products of few tiles: 64 x 64 tiles, 32 x 32 a wave, over a K
// range as the fast main loop takes it.
//
// A product of few 256 x 256 tiles leaves most CUs without work, and a large tile
// of few rows computes what nobody reads.  Here a tile is a sixteenth, a workgroup
// needs 34 KB of LDS and 152 registers, so that three of them share a CU, and four K
// steps of 256 values are in flight in registers, since one step computes for less
// than a load takes.  Sums run over K in the order of the plain product, so that
// the tile size does not show in a result.  Bound by latency, and by the caches
// where tiles are many: every operand byte is read four times as often as by the
// large tile.  With bias, GELU and residual, operands from memory: 64 x 4096 x 4096, 64
// tiles, 16 us (large tiles 33), 2048 x 2048 x 2048, 1024 tiles, 23 (31); from the caches
// 11 and 19.  (There, a wave taking every fourth K step of the whole tile, the partial
// sums added in LDS: 10 and 19, with 2048 tiles 32 against 25; fragments loaded straight
// to their lanes, 64 lines an instruction: 20.)
#pragma once

#include "gemm_epilogue.h"

namespace mx {

constexpr int kSmallTile = 64, kSmallThreads = 256;
constexpr int kSmallPitch = kSmallTile + 4;              // floats: an odd number of 16-byte chunks a row
// one stage: A codes, B codes (128 bytes a row), A scales, B scales (8 bytes a row)
constexpr int kSmallB = kSmallTile * BKB, kSmallScales = 2 * kSmallB, kSmallStage = kSmallScales + 2 * kSmallTile * 8;
constexpr int kSmallSmem = 2 * kSmallStage;
static_assert(kSmallTile * kSmallPitch * 4 <= kSmallSmem, "the tile's sums fit in the stages");

struct SmallOperand {
  __amdgpu_buffer_rsrc_t codes, scales;                  // from the tile's first row on
};

__device__ __forceinline__ SmallOperand small_operand(const Operand& x, int64_t row0, int64_t K) {
  const int64_t rows = min((int64_t)kSmallTile, x.rows - row0);
  return SmallOperand{buffer_rsrc(x.codes + row0 * (K >> 1), rows * (K >> 1)), buffer_rsrc(x.scales + row0 * (K >> 5), rows * (K >> 5))};
}

// A thread's share of a K step: chunk t & 7 of rows t / 8 and 32 + t / 8 of both
// operands, and the eight scale bytes of a row (wave 0: A's, wave 1: B's).
struct SmallStep {
  v4i a[2], b[2];
  uint2 scales;
};

// Rows past the operand and blocks outside the K range read as zero, their scales
// too: a scale byte of another row may stand for no number.  (The range check covers
// the lane offset, not the scalar one, which carries the K position.)
__device__ __forceinline__ void load_small(const SmallOperand& a, const SmallOperand& b, int64_t K, const KRange& kr, int step, int wave,
                                           SmallStep& x) {
  const int t = threadIdx.x, lsc = (int)(K >> 5);
  const uint32_t ldb = (uint32_t)(K >> 1), so = (uint32_t)step * BKB;
  const uint32_t v = (uint32_t)(8 * step + (t & 7) - kr.lo) < (uint32_t)kr.count ? (uint32_t)(t >> 3) * ldb + (t & 7) * 16 : kOffNone;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    x.a[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(a.codes, v + (uint32_t)(32 * j) * ldb, so, 0));
    x.b[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(b.codes, v + (uint32_t)(32 * j) * ldb, so, 0));
  }
  if (wave > 1) return;
  const __amdgpu_buffer_rsrc_t rs = wave ? b.scales : a.scales;
  const uint32_t vs = (uint32_t)((t & 63) * lsc);
  if (lsc >= 8) {
    // in a last, partial step the load is moved back to end with the row
    x.scales = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rs, vs, (uint32_t)min(8 * step, lsc - 8), 0));
  } else {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 8; ++q)
      w[q >> 2] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, q < lsc ? vs + (uint32_t)q : kOffNone, 0, 0) << (8 * (q & 3));
    x.scales = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ void write_small(uint8_t* stage, int64_t K, const KRange& kr, int step, int wave,
                                            const SmallStep& x) {
  const int t = threadIdx.x;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 32 * j + (t >> 3), at = row * BKB + swz(row, t & 7) * 16;
    *reinterpret_cast<v4i*>(stage + at) = x.a[j];
    *reinterpret_cast<v4i*>(stage + kSmallB + at) = x.b[j];
  }
  if (wave > 1) return;
  const int moved = K >= 256 ? max(8 * step - ((int)(K >> 5) - 8), 0) : 0;
  const int from = max(kr.lo - 8 * step, 0), to = min(kr.lo + kr.count - 8 * step, 8);   // bytes of the range
  const uint64_t in = (~(uint64_t)0 << (8 * from)) & (~(uint64_t)0 >> (8 * (8 - to)));
  *reinterpret_cast<uint64_t*>(stage + kSmallScales + 8 * t) = (__builtin_bit_cast(uint64_t, x.scales) >> (8 * moved)) & in;
}

template <int S>
__device__ __forceinline__ void mfma_small(const uint8_t* stage, int ra, int rb, int h, uint32_t sa, uint32_t sb, v16f& acc) {
  const v4i a = *reinterpret_cast<const v4i*>(stage + ra * BKB + swz(ra, 4 * h + S) * 16);
  const v4i b = *reinterpret_cast<const v4i*>(stage + kSmallB + rb * BKB + swz(rb, 4 * h + S) * 16);
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(widen(b), widen(a), acc, 4, 4, S, (int)sb, S, (int)sa);
}

// Tile (m0, n0): rows up to A.rows, columns up to B.rows (a multiple of 32).  A2,
// B2: a second pair of the same shapes, whose K steps follow; or null codes.
// Rows are K long, of which the range kr is taken; one of no steps gives zeros.
template <bool PLAIN>
__device__ __forceinline__ void small_tile(float* smem, const Operand& A, const Operand& B, const Operand& A2, const Operand& B2,
                                           int64_t m0, int64_t n0, int64_t K, const KRange& kr, const Epilogue& e) {
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  const int r = lane & 31, hl = lane >> 5, ra = 32 * (wave >> 1) + r, rb = 32 * (wave & 1) + r;
  const int nk1 = kr.steps, nk = A2.codes ? 2 * nk1 : nk1;
  const int64_t M = A.rows, N = B.rows;
  v16f acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.0f;
  if (nk > 0) {
    const SmallOperand a1 = small_operand(A, m0, K), b1 = small_operand(B, n0, K);
    const SmallOperand a2 = A2.codes ? small_operand(A2, m0, K) : a1, b2 = A2.codes ? small_operand(B2, n0, K) : b1;
    uint8_t* const lds = reinterpret_cast<uint8_t*>(smem);
    SmallStep x[4];
    const auto load = [&](int s, SmallStep& y) {
      if (s >= nk) return;
      const bool second = s >= nk1;
      load_small(second ? a2 : a1, second ? b2 : b1, K, kr, kr.first + (second ? s - nk1 : s), wave, y);
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) load(u, x[u]);
    // One barrier a step: it waits for this wave's LDS accesses, so a stage is
    // written again only when all waves have read it, two steps later.
    for (int s0 = 0; s0 < nk; s0 += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = s0 + u;
        if (s >= nk) break;
        uint8_t* const stage = lds + (u & 1) * kSmallStage;
        write_small(stage, K, kr, kr.first + (s >= nk1 ? s - nk1 : s), wave, x[u]);
        load(s + 4, x[u]);
        pp_sync();
        const uint32_t sa = *reinterpret_cast<const uint32_t*>(stage + kSmallScales + 8 * ra + 4 * hl);
        const uint32_t sb = *reinterpret_cast<const uint32_t*>(stage + kSmallScales + 8 * (kSmallTile + rb) + 4 * hl);
        mfma_small<0>(stage, ra, rb, hl, sa, sb, acc);
        mfma_small<1>(stage, ra, rb, hl, sa, sb, acc);
        mfma_small<2>(stage, ra, rb, hl, sa, sb, acc);
        mfma_small<3>(stage, ra, rb, hl, sa, sb, acc);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<float4*>(smem + ra * kSmallPitch + 32 * (wave & 1) + 8 * g + 4 * hl) =
        make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
  __syncthreads();
  const int ch = threadIdx.x & 7;
  const int64_t col = n0 + 8 * ch;
  if (col >= N) return;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int in = 32 * pass + (threadIdx.x >> 3);
    const int64_t row = m0 + in;
    if (row >= M) return;
    const float4* const p = reinterpret_cast<const float4*>(smem + in * kSmallPitch + 8 * ch);
    const float4 lo = p[0], hi = p[1];
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if constexpr (!PLAIN) {
      if (e.bias) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = __fadd_rn(v[u], e.bias_f32 ? static_cast<const float*>(e.bias)[col + u]
                                            : bf16_bits_to_f32(static_cast<const uint16_t*>(e.bias)[col + u]));
      }
      float res[8];
      if (e.residual) unpack8(*reinterpret_cast<const uint4*>(e.residual + row * e.ldr + col), res);
      if (e.z) put_row(e.z + row * N + col, v, 0);
      if (e.act != FP4_ACT_NONE)
        with_act(e.act, [&](auto act) {
          const auto apply = [&](auto fine) {
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = act_value<act(), fine()>(v[u]);
          };
          if (act() == FP4_ACT_GELU && e.y_f32) apply(std::true_type{});   // the others are the same for both
          else apply(std::false_type{});
        });
      if (e.residual) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __fadd_rn(v[u], res[u]);
      }
    }
    if (e.y_f32) {
      float* const q = static_cast<float*>(e.y) + row * e.ldy + col;
      if (PLAIN && e.accumulate) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = __fadd_rn(q[u], v[u]);
      }
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      put_row(static_cast<uint16_t*>(e.y) + row * e.ldy + col, v, 0);
    }
  }
}

}  // namespace mx
