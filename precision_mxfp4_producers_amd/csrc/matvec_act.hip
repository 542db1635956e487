// Few-row products with bias, activation and residual in their epilogue
// (fp4_matvec_act).
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.2 (Eq. 1) decode,
// §2.4 row layouts.
//
// Bound by the weights' way from memory, and where they are few by the start, x's
// way to LDS, the decode and the meeting of the sums: one row of 4096 x 14336
// (31 MB) 11 us, a bare loop of its loads 7.2; of 14336 x 4096 10.3; of 57344
// x 8192 (250 MB) 54, 4.6 TB/s; without products behind the loads 1 to 2 us less.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "matvec_core.h"

namespace mx {

template <int XT, int MT, int NT, int NW, int U, bool STAGED, int SC>
__global__ __launch_bounds__(NW * 64) void matvec_act_kernel(MatvecArgs a, MvPlan plan, MvEpilogue e) {
  matvec_body<XT, kMx, MT, NT, NW, U, false, STAGED, SC, true>(a, plan, e);
}

// The epilogue of an empty reduction or one of a few weights.
template <int XT>
__global__ __launch_bounds__(256) void matvec_act_small_kernel(MatvecArgs a, MvEpilogue e) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.m * a.n; i += (int64_t)gridDim.x * 256)
    put_epilogue(e, (int)(i / a.n), i % a.n, small_sum<XT>(a, i / a.n, i % a.n));
}

template <int XT>
static fp4_status matvec_act_launch(const MatvecArgs& a, const MvEpilogue& e, hipStream_t stream) {
  if (a.n * (a.k / 32) < 4) {
    const int64_t grid = std::min<int64_t>((a.m * a.n + 255) / 256, 65536);
    hipLaunchKernelGGL(matvec_act_small_kernel<XT>, dim3((unsigned)grid), dim3(256), 0, stream, a, e);
    return launch_status();
  }
  matvec_variant<kMx, false, kWordScales>(a, kMatvecGrid, [&](auto v, const MvPlan& plan, unsigned grid) {
    using V = decltype(v);
    hipLaunchKernelGGL((matvec_act_kernel<XT, V::MT, V::NT, V::NW, V::U, V::STAGED, V::SC>), dim3(grid),
                       dim3(V::NW * 64), 0, stream, a, plan, e);
  });
  return launch_status();
}

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_matvec_act(int64_t m, int64_t n, int64_t k, const void* x, int64_t ldx, const uint8_t* x_scales,
                          const uint8_t* w_codes, const uint8_t* w_scales, const void* bias, fp4_dtype bias_type,
                          fp4_act act, const uint16_t* residual, int64_t ldr, void* y, fp4_dtype y_type, int64_t ldy,
                          hipStream_t stream) {
  if (!dtype_ok(bias_type) || !dtype_ok(y_type) || act < FP4_ACT_NONE || act > FP4_ACT_SILU) return FP4_EINVAL;
  const bool e4m3 = x_scales != nullptr, f32 = y_type == FP4_F32;
  if (ldy < n || (residual && ldr < n) || (e4m3 && ldx != k)) return FP4_ESHAPE;
  const fp4_status st = matvec_check(m, n, k, x, ldx, x_scales, e4m3, w_codes, w_scales, y);
  if (st != FP4_OK || m == 0 || n == 0) return st;
  if ((reinterpret_cast<uintptr_t>(y) & (f32 ? 3 : 1)) || (reinterpret_cast<uintptr_t>(residual) & 1) ||
      (reinterpret_cast<uintptr_t>(bias) & (bias_type == FP4_F32 ? 3 : 1)))
    return FP4_EALIGN;
  const MatvecArgs a{(int)m, n, k, x, ldx, x_scales, w_codes, w_scales, nullptr, 0, nullptr, 0, 0, nullptr};
  const MvEpilogue e{bias, residual, ldr, y, ldy, (int)act, bias_type == FP4_F32, f32};
  return e4m3 ? matvec_act_launch<kXE4m3>(a, e, as_stream(stream)) : matvec_act_launch<kXBf16>(a, e, as_stream(stream));
}

}  // extern "C"
