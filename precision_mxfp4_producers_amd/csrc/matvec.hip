// Products of a few rows of activations with 4-bit weights under group scales:
// fp4_matvec (MXFP4 weights), fp4_nv_matvec (CTA-local NVFP4 weights) and
// fp4_swiglu_matvec (the gated FFN's first half).  The single-token and
// small-batch form of fp4_gemm, fp4_nv_gemm and fp4_swiglu_producer: the
// weights are the row layouts that the training step's weight producers emit,
// the activations stay in bf16 or come as the E4M3 codes of
// fp4_rmsnorm_producer.
//
// The decoded weights are exact in bf16, so that the products run on the bf16
// matrix cores with fp32 sums, 4e-8 from float64 in the 2-norm (the scaled
// 8-bit by 4-bit products were 4e-6 from it after 32 steps).
//
// Bound by HBM for few rows: 57344 x 8192 MXFP4 with five E4M3 rows, 250 MB,
// 49 us (5.1 TB/s; a bare loop of the same loads takes 41, contiguous loads
// 34); gate/up 14336 x 4096 with one row, 62 MB, 13.7 us (calls in a row; some 1
// us more in a kernel trace); 4096 x 4096 with one row, 9 MB, 4.8 us (kernel
// trace; a bare loop 3.8).  With more rows x's way through LDS takes over:
// gate/up 14336 x 4096 with 16 rows 16.4 us, 4096 x 14336 NVFP4 with 33 rows 22.
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.2 (Eq. 1) decode,
// §2.4 row layouts, §3.2 gated FFN.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "mx_device.h"

namespace mx {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Weight encodings and activation types.
constexpr int kMx = 0, kNv = 1;
constexpr int kXBf16 = 0, kXE4m3 = 1;

struct MatvecArgs {
  int m;                                                 // rows of x
  int64_t n, k;                                          // rows of W (of W1 for the gated form), their length
  const void* x;                                         // bf16 [m][ldx], or E4M3 codes [m][k]
  int64_t ldx;
  const uint8_t* x_scales;                               // E8M0 [m][k/32] (E4M3 codes)
  const uint8_t* codes;                                  // [n][k/2] (gated: [2n][k/2])
  const uint8_t* scales;                                 // [n][k/32] E8M0 or [n][k/16] E4M3
  const float* factors;                                  // NVFP4: factors[(row / 256) * factor_stride]
  int64_t factor_stride;
  float* c;                                              // [m][ldc]
  int64_t ldc;
  int accumulate;
  uint16_t* h;                                           // gated: [m][n]
};

// Eight E2M1 codes -> eight bf16 values times their group scale (MXFP4: a power
// of two, of which the converter reads the exponent field; NVFP4: the value of
// an E4M3 byte), exact: E2M1 has 2 significant bits, with an E4M3 scale the
// product has 6.
template <int WT>
__device__ __forceinline__ bf16x8_t decode8(uint32_t w, float s) {
  bf16x2_t p[4];
  if constexpr (WT == kMx) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x2_t v;
      if (j == 0) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
      else if (j == 1) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
      else if (j == 2) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
      else v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
      p[j] = bf16x2_t{(__bf16)__fmul_rn(v[0], s), (__bf16)__fmul_rn(v[1], s)};
    }
  }
  return bf16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// Each of these exchanges a register bit (a: 0, b: 1) with one bit of the lane
// index: afterwards a lane whose bit is 0 holds its own a and its partner's a,
// one whose bit is 1 its partner's b and its own b.
__device__ __forceinline__ void exchange_bit5(uint32_t& a, uint32_t& b) {
  const auto v = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = v[0]; b = v[1];
}
__device__ __forceinline__ void exchange_bit4(uint32_t& a, uint32_t& b) {
  const auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = v[0]; b = v[1];
}
// Two such exchanges with bit BIT (0 or 1: the partner is in the quad): one
// conditional move a result, its other operand read across the quad, which the
// compiler makes two of.  low: the lanes whose bit is 0.  The nop covers the
// two cycles that a lane-crossing read needs behind a write of its source.
template <int BIT>
__device__ __forceinline__ void exchange_quad(uint32_t& a0, uint32_t& b0, uint32_t& a1, uint32_t& b1) {
  constexpr uint64_t low = BIT == 0 ? 0x5555555555555555ull : 0x3333333333333333ull;
  uint32_t oa0, ob0, oa1, ob1;
#define MX_QUAD(PERM)                                                                  \
  asm("s_nop 1\n\t"                                                                    \
      "s_mov_b64 vcc, %8\n\t"                                                          \
      "v_cndmask_b32_dpp %0, %5, %4, vcc quad_perm:" PERM " row_mask:0xf bank_mask:0xf\n\t" \
      "v_cndmask_b32_dpp %2, %7, %6, vcc quad_perm:" PERM " row_mask:0xf bank_mask:0xf\n\t" \
      "s_not_b64 vcc, vcc\n\t"                                                         \
      "v_cndmask_b32_dpp %1, %4, %5, vcc quad_perm:" PERM " row_mask:0xf bank_mask:0xf\n\t" \
      "v_cndmask_b32_dpp %3, %6, %7, vcc quad_perm:" PERM " row_mask:0xf bank_mask:0xf"     \
      : "=&v"(oa0), "=&v"(ob0), "=&v"(oa1), "=&v"(ob1)                                 \
      : "v"(a0), "v"(b0), "v"(a1), "v"(b1), "s"(low)                                   \
      : "vcc", "scc")
  if constexpr (BIT == 0) MX_QUAD("[1,0,3,2]");
  else MX_QUAD("[2,3,0,1]");
#undef MX_QUAD
  a0 = oa0; b0 = ob0; a1 = oa1; b1 = ob1;
}

// Byte Q of a word as an E8M0 scale: its bits at the exponent's place.
template <int Q>
__device__ __forceinline__ float e8m0_byte(uint32_t w) {
  uint32_t o;
  const uint32_t sh = 23;
#define MX_BYTE(SEL)                                                                                      \
  asm("v_lshlrev_b32_sdwa %0, %1, %2 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:DWORD src1_sel:" SEL \
      : "=v"(o)                                                                                           \
      : "v"(sh), "v"(w))
  if constexpr (Q == 0) MX_BYTE("BYTE_0");
  else if constexpr (Q == 1) MX_BYTE("BYTE_1");
  else if constexpr (Q == 2) MX_BYTE("BYTE_2");
  else MX_BYTE("BYTE_3");
#undef MX_BYTE
  return __uint_as_float(o);
}

// The codes of a step as loaded, lane 4 rho + c holding 16-byte piece c of a
// row, to the products' operand: word q of lane 16 g + r becomes word g of
// piece q of row r, rho = 4 (r & 3) + (r >> 2).  The four lanes of a row load
// 64 consecutive bytes: the address unit takes four neighbouring lanes at a
// time, and loads laid out as the operand (neighbouring lanes: different rows)
// took four times as long even from the L1.
__device__ __forceinline__ void to_operand(uint32_t (&c)[4]) {
  exchange_bit5(c[0], c[2]);
  exchange_bit5(c[1], c[3]);
  exchange_bit4(c[0], c[1]);
  exchange_bit4(c[2], c[3]);
  exchange_quad<1>(c[0], c[2], c[1], c[3]);
  exchange_quad<0>(c[0], c[1], c[2], c[3]);
}

// Sixteen E4M3 codes with one E8M0 scale -> two fragments of eight bf16 values.
__device__ __forceinline__ void decode_x16(const v4i w, uint32_t sc, bf16x8_t& a, bf16x8_t& b) {
  const float s = __uint_as_float(sc << 23);
  bf16x2_t p[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    p[2 * q] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q], s, false);
    p[2 * q + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q], s, true);
  }
  a = bf16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  b = bf16x8_t{p[4][0], p[4][1], p[5][0], p[5][1], p[6][0], p[6][1], p[7][0], p[7][1]};
}

// NW waves form a workgroup: sixteen, or eight for more than one tile of x
// rows, whose operands take the registers of two waves.  A tile is 16 rows of
// W (gated: 8 of W1 and the same 8 of W3).  KW waves share NT tiles (one, or
// two) and split K; the workgroup works on NW / KW such sets at a time and
// walks groups of them blockIdx.x, blockIdx.x + gridDim.x, ...
//
// A step is 128 values of K; product q = 0 .. 3 of its four 16x16x32 bf16
// products takes values 32 q + 8 g .. + 7 in lane (r = lane & 15, g = lane >>
// 4), row r of W and of x.  An item is U consecutive
// steps; wave kw takes items kw, kw + KW, ... of a tile, and the loads of its
// next item, across the end of a tile too, are in flight during the products
// of the current one.  No branch surrounds a load: the compiler could not
// count the outstanding ones and would wait for all.  The partial sums meet in
// LDS and are added in wave order: deterministic, no atomics, no workspace.
//
// x goes through LDS as bf16: all of it once per workgroup where it fits
// (STAGED), else each wave brings its own steps, with the item, into a room of
// its own (no barrier between waves; wave_lds_order between its writes and
// its reads).
// WHOLE: K is a multiple of U steps and the scales are aligned to words, so
// that the scale bytes of an item come with one load, spread like the codes,
// and reach the other lanes of a row by permutes.
constexpr int kLds = 160 * 1024;
constexpr int kStageBytes = 143 * 1024;                  // most of x in LDS; the rest is the partial sums'
constexpr int kXPitch = 256 + 64;                        // of a wave's own step of x
// A wave's own room: 16 MT rows of a step; its partial sums take the same place.
__host__ __device__ constexpr int room_bytes(int mt) { return 16 * mt * kXPitch; }

// Bytes between staged rows of x: 64 past the rounded row.  An operand's four
// lane groups read 64 consecutive bytes of a row, so that four rows fill the 64
// banks (16 bytes more a row left 4 of 9 LDS cycles to bank conflicts).
__host__ __device__ constexpr int64_t stage_pitch(int64_t k) { return (k + 127) / 128 * 256 + 64; }

// How a launch splits the work (host side).
struct MvPlan {
  int kw_log2;                                           // waves per tile
  int batch;                                             // groups of tiles between two meetings of the partial sums
};

// Words of a row's scale bytes in an item of U steps.
template <int WT, int U>
constexpr int kScaleWords = WT == kMx ? U : 2 * U;

// One item of W as loaded: pieces of codes, and one word of a row's scale
// bytes; of a partial step the four bytes that this lane's products take.
template <int WT, int NT, int U, bool WHOLE>
struct MvItem {
  v4i c[NT][U];
  uint32_t s[NT][WHOLE ? 1 : 4];
};

// One step of x, as loaded: sixteen bytes a lane, 16 (bf16) or 8 (E4M3) lanes a row.
template <int XT, int MT>
struct MvX {
  v4i v[XT == kXBf16 ? 4 * MT : 2 * MT];
  uint32_t s[2 * MT];
};

// Waits for this wave's LDS accesses and meets the workgroup's other waves;
// global loads stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// The same without the wait; the compiler moves no access across it.
__device__ __forceinline__ void wave_barrier() { asm volatile("s_barrier" ::: "memory"); }
// Between LDS accesses of one wave whose lanes read what others wrote: the
// hardware keeps a wave's LDS accesses in order, and this the compiler, which
// sees a thread's own addresses only and may take them for distinct.  It makes
// no instruction.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
}

template <int XT, int WT, int MT, int NT, int NW, int U, bool GATE, bool STAGED, bool WHOLE>
__global__ __launch_bounds__(NW * 64) void matvec_kernel(MatvecArgs a, MvPlan plan) {
  static_assert(!STAGED || (MT == 1 && NT == 1), "sixteen rows of x and one tile at a time");
  static_assert((WHOLE && STAGED) || U == 1, "a partial step, and one that brings its x, is an item of its own");
  constexpr int ROWS = GATE ? 8 : 16;                    // output columns of a tile
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  constexpr int kWaveFloats = STAGED ? 260 : room_bytes(MT) / 4;   // between two waves' partial sums
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // the staged x behind the partial sums; or this wave's room
  uint8_t* const stage = lds + (STAGED ? (uint32_t)plan.batch * (NW * kWaveFloats * 4) : (uint32_t)wave * room_bytes(MT));
  const int kw = wave & ((1 << plan.kw_log2) - 1), rt = wave >> plan.kw_log2, RT = NW >> plan.kw_log2;
  const int64_t kc = a.k >> 1, ks = a.k >> (WT == kMx ? 5 : 4);   // bytes of a row's codes and scales
  const int steps = (int)((a.k + 127) >> 7), items = (steps + U - 1) / U;
  const int per = (items + (1 << plan.kw_log2) - 1) >> plan.kw_log2;   // turns of a wave per tile
  const int64_t groups = (a.n + ROWS * NT * RT - 1) / (ROWS * NT * RT);
  const __amdgpu_buffer_rsrc_t rx =
      buffer_rsrc(a.x, XT == kXBf16 ? ((a.m - 1) * a.ldx + a.k) * 2 : (int64_t)a.m * a.k);
  const __amdgpu_buffer_rsrc_t rxs = buffer_rsrc(a.x_scales, XT == kXBf16 ? 0 : (int64_t)a.m * (a.k >> 5));

  // Workgroups that read x from L2 start at different places of K: their
  // requests would otherwise meet in the few channels that hold one place of
  // every row (rows of x lie a multiple of 4 KB apart).
  const int turned = STAGED ? 0 : (int)(blockIdx.x * 7u % (uint32_t)items);
  // Place in K of the wave's item of a turn (a wave that has none takes the last).
  const auto item_of = [&](int turn) {
    const int it = std::min(kw + (turn << plan.kw_log2), items - 1) + turned;
    return it < items ? it : it - items;
  };
  // A row past the end reads the last one (its sums are not stored).
  const auto row_of = [&](int64_t group, int j, int r) {
    return std::min(((group * RT + rt) * NT + j) * ROWS + (r & (ROWS - 1)), a.n - 1) + (GATE && r >= ROWS ? a.n : 0);
  };
  const auto load_w = [&](MvItem<WT, NT, U, WHOLE>& it, int64_t group, int turn) {
    const int item = item_of(turn), piece = lane & 3;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t row = row_of(group, j, 4 * ((lane >> 2) & 3) + (lane >> 4));
      const uint8_t* const c = a.codes + row * kc;
      if constexpr (WHOLE) {
#pragma unroll
        for (int u = 0; u < U; ++u) it.c[j][u] = *reinterpret_cast<const v4i*>(c + (item * U + u) * 64 + piece * 16);
        constexpr int D = kScaleWords<WT, U>;
        it.s[j][0] = reinterpret_cast<const uint32_t*>(a.scales + row * ks)[item * D + (piece & (D - 1))];
      } else {
        const int blocks = (int)(a.k >> 5), kb = item * 4;   // a block of 32 values is whole or absent
        const uint8_t* const s = a.scales + row_of(group, j, r) * ks;
        const v4i v = *reinterpret_cast<const v4i*>(c + std::min(kb + piece, blocks - 1) * 16);
        it.c[j][0] = kb + piece < blocks ? v : v4i{0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = std::min(kb + q, blocks - 1);
          it.s[j][q] = WT == kMx ? s[at] : s[2 * at + (g >> 1)];
        }
      }
    }
  };
  const auto load_x = [&](MvX<XT, MT>& it, int turn) {
    if constexpr (XT == kXBf16) {
      const uint32_t at = (uint32_t)item_of(turn) * 128 + 8 * (lane & 15);
#pragma unroll
      for (int j = 0; j < 4 * MT; ++j) {
        const int row = 4 * j + (lane >> 4);
        const uint32_t off = row < a.m && at < (uint32_t)a.k ? ((uint32_t)row * (uint32_t)a.ldx + at) * 2 : kOffNone;
        it.v[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, off, 0, 0));
      }
    } else {
      const uint32_t at = (uint32_t)item_of(turn) * 128 + 16 * (lane & 7);
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) {
        const int row = 8 * j + (lane >> 3);
        const bool ok = row < a.m && at < (uint32_t)a.k;
        it.v[j] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? (uint32_t)row * (uint32_t)a.k + at : kOffNone, 0, 0));
        it.s[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
            rxs, ok ? (uint32_t)row * (uint32_t)(a.k >> 5) + (at >> 5) : kOffNone, 0, 0);
      }
    }
  };
  // this step of x into the wave's room
  const auto put_x = [&](const MvX<XT, MT>& it) {
    if constexpr (XT == kXBf16) {
#pragma unroll
      for (int j = 0; j < 4 * MT; ++j)
        *reinterpret_cast<v4i*>(stage + (4 * j + (lane >> 4)) * kXPitch + (lane & 15) * 16) = it.v[j];
    } else {
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) {
        bf16x8_t lo, hi;
        decode_x16(it.v[j], it.s[j], lo, hi);
        bf16x8_t* const p = reinterpret_cast<bf16x8_t*>(stage + (8 * j + (lane >> 3)) * kXPitch + (lane & 7) * 32);
        p[0] = lo;
        p[1] = hi;
      }
    }
  };

  v4f acc[MT][NT];
  const uint32_t xrow = (STAGED ? (uint32_t)(r < a.m ? r : 0) * (uint32_t)stage_pitch(a.k) : (uint32_t)r * kXPitch) + g * 16;
  const auto multiply = [&](const MvItem<WT, NT, U, WHOLE>& it, int turn) {
    if (kw + (turn << plan.kw_log2) >= items) return;    // wave-uniform
    const int item = item_of(turn);
    // the item's scale words of this lane's row r, from the lanes that loaded the row
    uint32_t sw[NT][kScaleWords<WT, U>];
    if constexpr (WHOLE)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int d = 0; d < kScaleWords<WT, U>; ++d)
          sw[j][d] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (4 * (4 * (r & 3) + (r >> 2)) + d), (int)it.s[j][0]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bf16x8_t w[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v4i cw = it.c[j][u];
        uint32_t c[4] = {(uint32_t)cw[0], (uint32_t)cw[1], (uint32_t)cw[2], (uint32_t)cw[3]};
        to_operand(c);
        float sc[4];                                     // the scale of product q's values
        if constexpr (WT == kMx && WHOLE) {
          sc[0] = e8m0_byte<0>(sw[j][u]);
          sc[1] = e8m0_byte<1>(sw[j][u]);
          sc[2] = e8m0_byte<2>(sw[j][u]);
          sc[3] = e8m0_byte<3>(sw[j][u]);
        } else if constexpr (WT == kMx) {
#pragma unroll
          for (int q = 0; q < 4; ++q) sc[q] = __uint_as_float(it.s[j][q] << 23);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t b = WHOLE ? (sw[j][2 * u + (q >> 1)] >> (16 * (q & 1) + 8 * (g >> 1))) & 0xFFu : it.s[j][q];
            const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, 1.0f, false);
            sc[q] = d[0];
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) w[j][q] = decode8<WT>(c[q], sc[q]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint8_t* const x = stage + xrow + (STAGED ? (uint32_t)(item * U + u) * 256 : (uint32_t)i * 16 * kXPitch);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t xq = *reinterpret_cast<const bf16x8_t*>(x + 64 * q);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[j][q], xq, acc[i][j], 0, 0, 0);
        }
      }
    }
  };
  // Lane l of a partial tile holds rows 4 (l >> 4) .. + 3 of W against row l &
  // 15 of x.  Four partial sums a thread, then the threads of one sum (KW / 4
  // neighbouring lanes, in lane order); gated: the sums of a and b lie in
  // neighbouring groups of lanes.
  const float* const rf = reinterpret_cast<const float*>(lds);
  const auto finish = [&](int64_t group, int slots) {     // group: the first one since the last meeting
    lds_barrier();
    const int split = plan.kw_log2 - 2, sums = 16 * NT * a.m;   // of a wave's tiles: 16 NT rows of W, m rows of x
    const int count = (slots * RT * sums) << split;
    for (int e0 = wave * 64; e0 < count; e0 += NW * 64) {
      const int e = e0 + lane, part = e & ((1 << split) - 1);
      int q = std::min(e >> split, slots * RT * sums - 1);   // a last wave's spare lanes repeat the last sum
      const int ab = GATE ? q & 1 : 0;
      if (GATE) q >>= 1;
      const int nl = q & (ROWS - 1);
      q /= ROWS;
      const int j = q & (NT - 1);
      q /= NT;
      const int mr = (int)((uint32_t)q % (uint32_t)a.m);
      q = (int)((uint32_t)q / (uint32_t)a.m);
      const int t = q & (RT - 1), slot = q / RT, wr = nl + ROWS * ab;
      const float* const p = rf + (slot * NW + (t << plan.kw_log2) + 4 * part) * kWaveFloats + ((mr >> 4) * NT + j) * 256 +
                             ((wr >> 2) * 16 + (mr & 15)) * 4 + (wr & 3);
      float v = __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[kWaveFloats]), p[2 * kWaveFloats]), p[3 * kWaveFloats]);
      for (int s = 1; s < 1 << split; s <<= 1) v = __fadd_rn(v, __shfl_xor(v, s, 64));
      const int64_t row = (((group + (int64_t)slot * gridDim.x) * RT + t) * NT + j) * ROWS + nl;
      if constexpr (GATE) {
        const float other = __shfl_xor(v, 1 << split, 64);
        const uint32_t both = ab ? bf16_pack2_rne(other, v) : bf16_pack2_rne(v, other);   // a low, b high
        const float av[1] = {__uint_as_float(both << 16)};
        float sig[1], sl[1];
        sigmoid_silu_n(av, sig, sl);
        if (e < count && part == 0 && ab == 0 && row < a.n)
          a.h[mr * a.n + row] = (uint16_t)bf16_pack2_rne(__fmul_rn(sl[0], __uint_as_float(both & 0xFFFF0000u)), 0.0f);
      } else if (e < count && part == 0 && row < a.n) {
        if constexpr (WT == kNv) v = __fmul_rn(a.factors[(row >> 8) * a.factor_stride], v);
        float* const c = a.c + mr * a.ldc + row;
        *c = a.accumulate ? __fadd_rn(*c, v) : v;
      }
    }
    // the partial sums' room is free again once all have read (STAGED: the next item's barrier says so)
    if constexpr (!STAGED) lds_barrier();
  };

  // The workgroup's items in order: (group, turn), the same count for every
  // wave, so that all reach the barriers.
  const int64_t first = blockIdx.x;
  int64_t left = (groups - first + gridDim.x - 1) / gridDim.x * per;
  int64_t group = first;                                 // of the current item
  int turn = 0, slots = 0;
  const auto step = [&](int64_t& gr, int& tn) {
    if (++tn == per) { tn = 0; gr += gridDim.x; }
  };
  using W = MvItem<WT, NT, U, WHOLE>;
  MvX<XT, MT> x;                                         // the next step of x, on its way to the wave's room
  const auto ahead = [&](W& w) {                         // loads of the item after the current one
    int64_t gr = group;
    int tn = turn;
    step(gr, tn);
    load_w(w, gr, tn);
  };
  // The products of an item; at a tile's end its sums go to LDS.
  const auto use = [&](const W& w) {
    if constexpr (!STAGED) {
      int64_t gr = group;
      int tn = turn;
      step(gr, tn);
      wave_lds_order();                                  // the room: the last step's reads are before
      put_x(x);
      load_x(x, tn);
      wave_lds_order();                                  // its values: other lanes read them below
    }
    multiply(w, turn);
    // The waves keep together, so that their loads stay on neighbouring
    // addresses: left to drift, 57344 x 8192 took 54 us instead of 50, as it
    // did with more loads in flight.  Behind it all waves have read the sums of
    // the meeting before, whose place the ones below take.
    if constexpr (STAGED) wave_barrier();
    if (turn + 1 == per) {
      if constexpr (!STAGED) wave_lds_order();           // the sums take the room of the step just read
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          reinterpret_cast<v4f*>(lds)[(slots * NW + wave) * (kWaveFloats / 4) + (i * NT + j) * 64 + lane] = acc[i][j];
          acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
      ++slots;
    }
    step(group, turn);
  };
  // Stages x in chunks of eight values, zero past k: a thread takes every (64
  // NW)-th, B loads in flight.  W's first loads go out behind the first B, so
  // that waiting for those does not wait for these.
  const auto stage_x = [&](auto b, auto&& behind) {
    constexpr int B = b();
    const int chunks = steps * 16, drow = NW * 64 / chunks, dc = NW * 64 - drow * chunks;
    const uint32_t pitch = (uint32_t)stage_pitch(a.k);
    int row = (int)threadIdx.x / chunks, c = (int)threadIdx.x - row * chunks;
    const int passes = (a.m * chunks + NW * 64 * B - 1) / (NW * 64 * B);
    const auto pass = [&](auto&& then) {
      v4i v[B];
      uint32_t sc[B], at[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const bool ok = row < a.m && c * 8 < a.k;
        at[j] = row < a.m ? (uint32_t)row * pitch + c * 16 : 0xFFFFFFFFu;
        if constexpr (XT == kXBf16) {
          v[j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                             rx, ok ? ((uint32_t)row * (uint32_t)a.ldx + c * 8) * 2 : kOffNone, 0, 0));
        } else {
          typedef int v2i __attribute__((ext_vector_type(2)));
          const v2i y = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(
                                                    rx, ok ? (uint32_t)row * (uint32_t)a.k + c * 8 : kOffNone, 0, 0));
          v[j] = v4i{y.x, y.y, 0, 0};
          sc[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
              rxs, ok ? (uint32_t)row * (uint32_t)(a.k >> 5) + (c >> 2) : kOffNone, 0, 0);
        }
        c += dc;
        row += drow;
        if (c >= chunks) c -= chunks, ++row;
      }
      then();
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if constexpr (XT == kXE4m3) {
          bf16x8_t lo, unused;
          decode_x16(v[j], sc[j], lo, unused);
          v[j] = __builtin_bit_cast(v4i, lo);
        }
        if (at[j] != 0xFFFFFFFFu) *reinterpret_cast<v4i*>(stage + at[j]) = v[j];
      }
    };
    pass(behind);
    for (int p = 1; p < passes; ++p) pass([] {});
    lds_barrier();
  };
  const auto begin = [&](auto&& loads) {
    if constexpr (STAGED) {
      if (a.m * steps * 16 <= NW * 64) stage_x(std::integral_constant<int, 1>{}, loads);
      else stage_x(std::integral_constant<int, 8>{}, loads);
    } else {
      loads();
    }
  };
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  W w0, w1;
  begin([&] {
    load_w(w0, first, 0);
    if constexpr (!STAGED) load_x(x, 0);
  });
  if (left == 1) {                                       // a small product: one item a wave
    use(w0);
    finish(first, slots);
    return;
  }
  // One stretch of items up to a meeting of the sums, its first in p, in pairs
  // so that each item has registers of its own; true where it was odd: the next
  // item is in q then.  Loads past the last item go to the last row, unused.
  const int64_t stretch = (int64_t)plan.batch * per;
  const auto run = [&](W& p, W& q) {
    int64_t n = std::min(left, stretch);
    const int64_t met = group;
    left -= n;
    for (; n >= 2; n -= 2) {
      ahead(q);
      use(p);
      ahead(p);
      use(q);
    }
    if (n) {
      ahead(q);
      use(p);
    }
    finish(met, slots);
    slots = 0;
    return n != 0;
  };
  while (left > 0)
    if (run(w0, w1) && left > 0) run(w1, w0);
}

// C (+)= 0 for an empty reduction.
__global__ void matvec_zero_kernel(MatvecArgs a) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < a.m * a.n; e += (int64_t)gridDim.x * 256) {
    if (a.h) a.h[e] = 0;
    else a.c[(e / a.n) * a.ldc + e % a.n] = 0.0f;
  }
}

constexpr int kMatvecMaxM = 64;
constexpr int64_t kMatvecGrid = 256;                     // one workgroup of 16 waves per CU

template <int XT, int WT, bool GATE>
static fp4_status matvec_launch(const MatvecArgs& a, hipStream_t stream) {
  if (a.k == 0) {
    if (a.accumulate) return FP4_OK;
    const int64_t grid = std::min<int64_t>((a.m * a.n + 255) / 256, 65536);
    hipLaunchKernelGGL(matvec_zero_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a);
    return launch_status();
  }
  constexpr int ROWS = GATE ? 8 : 16;
  const int64_t tiles = (a.n + ROWS - 1) / ROWS, steps = (a.k + 127) / 128;
  const bool staged = a.m <= 16 && a.m * stage_pitch(a.k) <= kStageBytes;
  const int mt = (a.m + 15) / 16, nw = mt > 1 ? 8 : 16;
  // Where x is not staged its way through LDS bounds the kernel (110 cycles a
  // step and 16 rows): two tiles of W a wave share it, if there are as many for
  // every CU (8192 x 14336, one tile to two: 17 rows 26.6 to 20.4 us, 33 rows
  // 36.6 to 25.5, 64 rows 47.3 to 38.4, NVFP4 29.6 to 24.9, 38.3 to 29.3 and
  // 51.1 to 40.7; 16 rows MXFP4 20.3 to 17.5; NVFP4 lost, 20.3 to 21.5, and
  // keeps one).  So also where two tiles spill a few registers, bf16 x with
  // more than 48 rows, and gated with up to 16 (20.8 to 18.8).
  const bool words = (reinterpret_cast<uintptr_t>(a.scales) & 3) == 0, whole = a.k % 128 == 0 && words;
  const int nt = !staged && whole && tiles >= 2 * kMatvecGrid && (WT == kMx || mt > 1) ? 2 : 1;
  // groups of tiles between two meetings of the sums: what LDS holds beside x
  const int64_t slot = 16 * 260 * 4;
  const int batch = staged ? (int)std::min<int64_t>((kLds - a.m * stage_pitch(a.k)) / slot, 4) : 1;
  // Waves per tile and steps per item: the pair whose longest workgroup has
  // the fewest steps to walk, a meeting of the sums counted as one (both take
  // some 0.8 us; 16 rows on gate/up 14336 x 4096, whose x leaves room for one
  // group's sums: 20.7 us without counting them, 16.6 with); longer items
  // and fewer waves a tile where equal.
  int u = 1, kw = 4;
  int64_t best = INT64_MAX;
  const auto groups_of = [&](int log2) { return (tiles + nt * (nw >> log2) - 1) / (nt * (nw >> log2)); };
  constexpr int kMaxU = WT == kMx ? 4 : 2;               // what the registers hold
  for (int uu = staged ? kMaxU : 1; uu >= 1; uu >>= 1) {
    if (uu > 1 && (a.k % (128 * uu) != 0 || !words)) continue;
    for (int log2 = 2; log2 <= (nw == 16 ? 4 : 3); ++log2) {
      const int64_t rounds = (groups_of(log2) + kMatvecGrid - 1) / kMatvecGrid;
      const int64_t cost =
          rounds * (((steps + uu - 1) / uu + (1 << log2) - 1) >> log2) * uu + (rounds + batch - 1) / batch;
      if (cost < best) best = cost, u = uu, kw = log2;
    }
  }
  const MvPlan plan{kw, batch};
  const unsigned grid = (unsigned)std::min(groups_of(kw), kMatvecGrid);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(nw * 64), 0, stream, a, plan); };
  if (staged) {
    if (u == 2) go(matvec_kernel<XT, WT, 1, 1, 16, 2, GATE, true, true>);
    else if (u == 1 && whole) go(matvec_kernel<XT, WT, 1, 1, 16, 1, GATE, true, true>);
    else if (u == 1) go(matvec_kernel<XT, WT, 1, 1, 16, 1, GATE, true, false>);
    if constexpr (kMaxU == 4)
      if (u == 4) go(matvec_kernel<XT, WT, 1, 1, 16, 4, GATE, true, true>);
    return launch_status();
  }
  const auto own = [&](auto mtc) {                       // each wave brings its own steps of x
    constexpr int MT = mtc(), NW = MT > 1 ? 8 : 16;
    if constexpr (WT == kMx || MT > 1)
      if (nt == 2) return go(matvec_kernel<XT, WT, MT, 2, NW, 1, GATE, false, true>);
    whole ? go(matvec_kernel<XT, WT, MT, 1, NW, 1, GATE, false, true>)
          : go(matvec_kernel<XT, WT, MT, 1, NW, 1, GATE, false, false>);
  };
  if (mt == 1) own(std::integral_constant<int, 1>{});
  else if (mt == 2) own(std::integral_constant<int, 2>{});
  else if (mt == 3) own(std::integral_constant<int, 3>{});
  else own(std::integral_constant<int, 4>{});
  return launch_status();
}

// Checks shared by the three calls; n counts output columns, `stack` the rows
// of codes per output column.
static fp4_status matvec_check(int64_t m, int64_t n, int64_t k, const void* x, int64_t ldx, const uint8_t* x_scales,
                               bool e4m3, const uint8_t* codes, const uint8_t* scales, const void* out) {
  if (m < 0 || m > kMatvecMaxM || n < 0 || !mult32z(k) || k >= ((int64_t)1 << 24) || ldx < k ||
      ldx >= ((int64_t)1 << 24))
    return FP4_ESHAPE;
  if (m == 0 || n == 0) return FP4_OK;
  if (n > ((int64_t)1 << 34)) return FP4_ESHAPE;
  if (!out) return FP4_EINVAL;
  if (k > 0 && (!x || !codes || !scales || (e4m3 && !x_scales))) return FP4_EINVAL;
  if (k > 0 && (!aligned16(x) || !aligned16(codes) || (!e4m3 && ldx % 8 != 0))) return FP4_EALIGN;
  return FP4_OK;
}

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_matvec(int64_t m, int64_t n, int64_t k, const void* x, int64_t ldx, const uint8_t* x_scales,
                      const uint8_t* w_codes, const uint8_t* w_scales, float* c, int64_t ldc, int accumulate,
                      hipStream_t stream) {
  if (accumulate != 0 && accumulate != 1) return FP4_EINVAL;
  const bool e4m3 = x_scales != nullptr;
  if (ldc < n || (e4m3 && ldx != k)) return FP4_ESHAPE;
  const fp4_status st = matvec_check(m, n, k, x, ldx, x_scales, e4m3, w_codes, w_scales, c);
  if (st != FP4_OK || m == 0 || n == 0) return st;
  if (reinterpret_cast<uintptr_t>(c) & 3) return FP4_EALIGN;
  const MatvecArgs a{(int)m, n, k, x, ldx, x_scales, w_codes, w_scales, nullptr, 0, c, ldc, accumulate, nullptr};
  return e4m3 ? matvec_launch<kXE4m3, kMx, false>(a, as_stream(stream))
              : matvec_launch<kXBf16, kMx, false>(a, as_stream(stream));
}

fp4_status fp4_nv_matvec(int64_t m, int64_t n, int64_t k, const uint16_t* x, int64_t ldx, const uint8_t* w_codes,
                         const uint8_t* w_scales, const float* w_factors, int64_t w_factor_stride, float* c,
                         int64_t ldc, int accumulate, hipStream_t stream) {
  if ((accumulate != 0 && accumulate != 1) || w_factor_stride < 0) return FP4_EINVAL;
  if (ldc < n) return FP4_ESHAPE;
  const fp4_status st = matvec_check(m, n, k, x, ldx, nullptr, false, w_codes, w_scales, c);
  if (st != FP4_OK || m == 0 || n == 0) return st;
  if (k > 0 && !w_factors) return FP4_EINVAL;
  if ((reinterpret_cast<uintptr_t>(c) & 3) || (reinterpret_cast<uintptr_t>(w_factors) & 3)) return FP4_EALIGN;
  const MatvecArgs a{(int)m, n, k, x, ldx, nullptr, w_codes, w_scales, w_factors, w_factor_stride, c, ldc, accumulate,
                     nullptr};
  return matvec_launch<kXBf16, kNv, false>(a, as_stream(stream));
}

fp4_status fp4_swiglu_matvec(int64_t m, int64_t f, int64_t d, const void* x, int64_t ldx, const uint8_t* x_scales,
                             const uint8_t* w13_codes, const uint8_t* w13_scales, uint16_t* h, hipStream_t stream) {
  const bool e4m3 = x_scales != nullptr;
  if (e4m3 && ldx != d) return FP4_ESHAPE;
  const fp4_status st = matvec_check(m, f, d, x, ldx, x_scales, e4m3, w13_codes, w13_scales, h);
  if (st != FP4_OK || m == 0 || f == 0) return st;
  if (reinterpret_cast<uintptr_t>(h) & 1) return FP4_EALIGN;
  const MatvecArgs a{(int)m, f, d, x, ldx, x_scales, w13_codes, w13_scales, nullptr, 0, nullptr, 0, 0, h};
  return e4m3 ? matvec_launch<kXE4m3, kMx, true>(a, as_stream(stream))
              : matvec_launch<kXBf16, kMx, true>(a, as_stream(stream));
}

}  // extern "C"
