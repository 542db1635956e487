// Products of a few rows of activations with 4-bit weights under group scales:
// fp4_matvec (MXFP4 weights), fp4_nv_matvec (CTA-local NVFP4 weights) and
// fp4_swiglu_matvec (the gated FFN's first half).  The single-token and
// small-batch form of fp4_gemm, fp4_nv_gemm and fp4_swiglu_producer: the
// weights are the row layouts that the training step's weight producers emit,
// the activations stay in bf16 or come as the E4M3 codes of
// fp4_rmsnorm_producer.
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

// Four words of 32 E2M1 codes -> 32 bf16 values times their group scale(s),
// exact: E2M1 has 2 significant bits, with an E4M3 scale the product has 6.
template <int WT>
__device__ __forceinline__ void decode32(const v4i w, uint32_t sc, bf16x8_t (&o)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    bf16x2_t p[4];
    if constexpr (WT == kMx) {
      const float s = __uint_as_float(sc << 23);         // the converter reads the exponent field: 2^(byte - 127)
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], s, 0);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], s, 1);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], s, 2);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], s, 3);
    } else {
      const f32x2_t d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((q < 2 ? sc : sc >> 8) & 0xFFu, 1.0f, false);
      const float d = d2[0];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x2_t v;
        if (j == 0) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], 1.0f, 0);
        else if (j == 1) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], 1.0f, 1);
        else if (j == 2) v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], 1.0f, 2);
        else v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], 1.0f, 3);
        p[j] = bf16x2_t{(__bf16)__fmul_rn(v[0], d), (__bf16)__fmul_rn(v[1], d)};
      }
    }
    o[q] = bf16x8_t{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  }
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

// One workgroup computes 16 RT rows of W (gated: 16 RT rows of W1 and of W3)
// against all m <= 16 MT rows of x.  Its waves split K: wave w takes the
// 128-value steps w, w + NW, ...; lane (r = lane & 15, g = lane >> 4) holds
// values 32 g .. 32 g + 31 of the step of W row r and of x row r, which the
// 16x16x32 bf16 products take eight at a time (both operands list K in the
// same order).  The partial sums meet in LDS and are added in wave order:
// deterministic, no atomics, no workspace.
template <int XT, int WT, int MT, int RT, int NW, bool GATE>
__global__ __launch_bounds__(NW * 64) void matvec_kernel(MatvecArgs a) {
  constexpr int NT = GATE ? 2 * RT : RT;                 // 16-row tiles of W
  __shared__ v4f red[NW * MT * NT * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
  const int64_t kc = a.k >> 1, ks = a.k >> (WT == kMx ? 5 : 4);   // bytes of a row's codes and scales
  __amdgpu_buffer_rsrc_t rc[NT], rs[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t row = n0 + 16 * (GATE ? i >> 1 : i);
    const int64_t rows = std::max<int64_t>(0, std::min<int64_t>(16, a.n - row));
    const int64_t at = row + (GATE && (i & 1) ? a.n : 0);
    rc[i] = buffer_rsrc(a.codes + at * kc, rows * kc);
    rs[i] = buffer_rsrc(a.scales + at * ks, rows * ks);
  }
  const __amdgpu_buffer_rsrc_t rx =
      buffer_rsrc(a.x, XT == kXBf16 ? ((a.m - 1) * a.ldx + a.k) * 2 : (int64_t)a.m * a.k);
  const __amdgpu_buffer_rsrc_t rxs = buffer_rsrc(a.x_scales, XT == kXBf16 ? 0 : (int64_t)a.m * (a.k >> 5));
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (int)((a.k + 127) >> 7);
  for (int st = wave; st < steps; st += NW) {
    const uint32_t kb = (uint32_t)st * 4 + g;            // this lane's block of 32 values
    const bool in = kb * 32 < (uint32_t)a.k;             // k is a multiple of 32: a block is whole or absent
    bf16x8_t x[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = 16 * i + r;
      const bool ok = in && row < a.m;
      if constexpr (XT == kXBf16) {
        const uint32_t off = ok ? ((uint32_t)row * (uint32_t)a.ldx + kb * 32) * 2 : kOffNone;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          x[i][q] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16 * q, 0, 0));
      } else {
        const uint32_t off = ok ? (uint32_t)row * (uint32_t)a.k + kb * 32 : kOffNone;
        const uint32_t so = ok ? (uint32_t)row * (uint32_t)(a.k >> 5) + kb : kOffNone;
        const uint32_t sc = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rxs, so, 0, 0);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          decode_x16(__builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, off + 16 * q, 0, 0)), sc,
                     x[i][2 * q], x[i][2 * q + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t off = in ? (uint32_t)r * (uint32_t)kc + kb * 16 : kOffNone;
      const v4i w = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rc[j], off, 0, kLoadOnce));
      uint32_t sc;
      if constexpr (WT == kMx)
        sc = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs[j], in ? (uint32_t)r * (uint32_t)ks + kb : kOffNone, 0, 0);
      else
        sc = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[j], in ? (uint32_t)r * (uint32_t)ks + kb * 2 : kOffNone, 0, 0);
      bf16x8_t wf[4];
      decode32<WT>(w, sc, wf);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[q], x[i][q], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // lane l of a tile holds rows 4 (l >> 4) .. + 3 of W against row l & 15 of x
  const float* rf = reinterpret_cast<const float*>(red);
  const auto total = [&](int i, int j, int nl, int ml) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      v = __fadd_rn(v, rf[((((w * MT + i) * NT + j) * 64) + (nl >> 2) * 16 + ml) * 4 + (nl & 3)]);
    return v;
  };
  for (int e = threadIdx.x; e < MT * RT * 256; e += NW * 64) {
    const int tile = e >> 8, i = tile / RT, j = tile % RT, ml = (e >> 4) & 15, nl = e & 15;
    const int mr = 16 * i + ml;
    const int64_t row = n0 + 16 * j + nl;
    if (mr >= a.m || row >= a.n) continue;
    if constexpr (GATE) {
      const float av = bf16_bits_to_f32(f32_to_bf16_rne(total(i, 2 * j, nl, ml)));
      const float bv = bf16_bits_to_f32(f32_to_bf16_rne(total(i, 2 * j + 1, nl, ml)));
      float sig, s;
      sigmoid_silu(av, sig, s);
      a.h[mr * a.n + row] = (uint16_t)f32_to_bf16_rne(__fmul_rn(s, bv));
    } else {
      float v = total(i, j, nl, ml);
      if constexpr (WT == kNv) v = __fmul_rn(a.factors[(row >> 8) * a.factor_stride], v);
      float* p = a.c + mr * a.ldc + row;
      *p = a.accumulate ? __fadd_rn(*p, v) : v;
    }
  }
}

// C (+)= 0 for an empty reduction.
__global__ void matvec_zero_kernel(MatvecArgs a) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < a.m * a.n; e += (int64_t)gridDim.x * 256) {
    if (a.h) a.h[e] = 0;
    else a.c[(e / a.n) * a.ldc + e % a.n] = 0.0f;
  }
}

constexpr int kMatvecMaxM = 64;

template <int XT, int WT, bool GATE>
static fp4_status matvec_launch(const MatvecArgs& a, hipStream_t stream) {
  if (a.k == 0) {
    if (a.accumulate) return FP4_OK;
    const int64_t grid = std::min<int64_t>((a.m * a.n + 255) / 256, 65536);
    hipLaunchKernelGGL(matvec_zero_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a);
    return launch_status();
  }
  const auto go = [&](auto kernel, int rows, int nw) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.n + rows - 1) / rows)), dim3(nw * 64), 0, stream, a);
  };
  if (a.m <= 16) go(matvec_kernel<XT, WT, 1, 1, 8, GATE>, 16, 8);
  else if (a.m <= 32) go(matvec_kernel<XT, WT, 2, 1, 8, GATE>, 16, 8);
  else go(matvec_kernel<XT, WT, 4, 1, 8, GATE>, 16, 8);
  return launch_status();
}

// Checks shared by the three calls; n counts output columns, `stack` the rows
// of codes per output column.
static fp4_status matvec_check(int64_t m, int64_t n, int64_t k, const void* x, int64_t ldx, const uint8_t* x_scales,
                               bool e4m3, const uint8_t* codes, const uint8_t* scales, int64_t scale_align,
                               const void* out) {
  if (m < 0 || m > kMatvecMaxM || n < 0 || !mult32z(k) || k >= ((int64_t)1 << 24) || ldx < k ||
      ldx >= ((int64_t)1 << 24))
    return FP4_ESHAPE;
  if (m == 0 || n == 0) return FP4_OK;
  if (n > ((int64_t)1 << 34)) return FP4_ESHAPE;
  if (!out) return FP4_EINVAL;
  if (k > 0 && (!x || !codes || !scales || (e4m3 && !x_scales))) return FP4_EINVAL;
  if (k > 0 && (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & (scale_align - 1)) ||
                (!e4m3 && ldx % 8 != 0)))
    return FP4_EALIGN;
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
  const fp4_status st = matvec_check(m, n, k, x, ldx, x_scales, e4m3, w_codes, w_scales, 1, c);
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
  const fp4_status st = matvec_check(m, n, k, x, ldx, nullptr, false, w_codes, w_scales, 2, c);
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
  const fp4_status st = matvec_check(m, f, d, x, ldx, x_scales, e4m3, w13_codes, w13_scales, 1, h);
  if (st != FP4_OK || m == 0 || f == 0) return st;
  if (reinterpret_cast<uintptr_t>(h) & 1) return FP4_EALIGN;
  const MatvecArgs a{(int)m, f, d, x, ldx, x_scales, w13_codes, w13_scales, nullptr, 0, nullptr, 0, 0, h};
  return e4m3 ? matvec_launch<kXE4m3, kMx, true>(a, as_stream(stream))
              : matvec_launch<kXBf16, kMx, true>(a, as_stream(stream));
}

}  // extern "C"
