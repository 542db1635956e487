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
#include "matvec_core.h"

namespace mx {

template <int XT, int WT, int MT, int NT, int NW, int U, bool GATE, bool STAGED, bool WHOLE>
__global__ __launch_bounds__(NW * 64) void matvec_kernel(MatvecArgs a, MvPlan plan) {
  matvec_body<XT, WT, MT, NT, NW, U, GATE, STAGED, WHOLE ? kWholeScales : kByteScales, false>(a, plan, MvEpilogue{});
}

// C (+)= 0 for an empty reduction.
__global__ void matvec_zero_kernel(MatvecArgs a) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < a.m * a.n; e += (int64_t)gridDim.x * 256) {
    if (a.h) a.h[e] = 0;
    else a.c[(e / a.n) * a.ldc + e % a.n] = 0.0f;
  }
}

template <int XT, int WT, bool GATE>
static fp4_status matvec_launch(const MatvecArgs& a, hipStream_t stream) {
  if (a.k == 0) {
    if (a.accumulate) return FP4_OK;
    const int64_t grid = std::min<int64_t>((a.m * a.n + 255) / 256, 65536);
    hipLaunchKernelGGL(matvec_zero_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a);
    return launch_status();
  }
  matvec_variant<WT, GATE>(a, kMatvecGrid, [&](auto v, const MvPlan& plan, unsigned grid) {
    using V = decltype(v);
    hipLaunchKernelGGL((matvec_kernel<XT, WT, V::MT, V::NT, V::NW, V::U, GATE, V::STAGED, V::SC == kWholeScales>), dim3(grid),
                       dim3(V::NW * 64), 0, stream, a, plan);
  });
  return launch_status();
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
