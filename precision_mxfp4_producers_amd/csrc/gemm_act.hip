// Block-scaled E2M1 product with bias, activation and residual in its epilogue
// (fp4_gemm_act), on the fast main loop of the plain product.
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.3 (Eq. 4) for the
// product, §3.1 (a boundary leaves its consumer's operands without a round
// trip) for the epilogue.
//
// Bound by the matrix cores and, of the same workgroups, the store burst behind
// each tile (one workgroup a CU: nothing else runs beside it).  8192 x 14336 x
// 4096, 0.96 TFLOP, medians with operands from memory: 269 us with a bf16 y (3.6
// PFLOP/s; 296 with an fp32 one and a bias, the plain product 291), 312 with bias and z
// beside it, 308 with bias and GELU, 330 with all of them (2.9 PFLOP/s), 341 with bias
// and residual.  Products of few tiles take tiles of 64 x 64.
#include <hip/hip_runtime.h>

#include "abi_common.h"
#include "gemm_core.h"
#include "gemm_epilogue.h"
#include "gemm_small.h"

namespace mx {

template <int kMode>
__global__ __launch_bounds__(kFastThreads) void gemm_act_kernel(int64_t M, int64_t N, int64_t K,
                                                                const uint8_t* __restrict__ a_codes,
                                                                const uint8_t* __restrict__ a_scales,
                                                                const uint8_t* __restrict__ b_codes,
                                                                const uint8_t* __restrict__ b_scales, Epilogue e) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmemBytes];
  int64_t tm, tn;
  const int64_t tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN, pid = grid_tile();
  if (pid >= tiles_m * tiles_n) return;
  tile_coords_of(pid, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 2, wn = wave & 3, hl = lane >> 5;
  const Operand A{a_codes, a_scales, M}, B{b_codes, b_scales, N};
  v16f acc[4][2];
  if (kMode == kShort && K == 0) zero_tile(acc);          // z = bias
  else main_loop_fast<false, kMode>(smem, A, B, m0, n0, 0, K, acc, wm, wn, nullptr, nullptr, k_range(0, (int)(K >> 5)));
  store_epilogue<false>(smem, acc, e, M, N, m0, n0, wave, lane, wm, wn, hl);
}

__global__ __launch_bounds__(kSmallThreads, 3) void gemm_act_small_kernel(int64_t M, int64_t N, int64_t K,
                                                                       const uint8_t* __restrict__ a_codes,
                                                                       const uint8_t* __restrict__ a_scales,
                                                                       const uint8_t* __restrict__ b_codes,
                                                                       const uint8_t* __restrict__ b_scales, Epilogue e) {
  __shared__ __attribute__((aligned(16))) float smem[kSmallSmem / sizeof(float)];
  int64_t tm, tn;
  tile_coords((M + kSmallTile - 1) / kSmallTile, (N + kSmallTile - 1) / kSmallTile, tm, tn);
  const Operand A{a_codes, a_scales, M}, B{b_codes, b_scales, N}, none{};
  small_tile<false>(smem, A, B, none, none, tm * kSmallTile, tn * kSmallTile, K, k_range(0, (int)(K >> 5)), e);
}

// The most 64 x 64 tiles a product is given (large and small tiles, bias, GELU and
// residual, operands from memory: 300 x 1024 x 1024, 80 small tiles, 21 and 7.5 us; 512 x
// 2048 x 2048, 256, 30 and 11.5; 256 x 4096 x 14336, 256, 121 and 39; 1024 x 4096 x 4096,
// 1024, 45 and 36; 1024 x 4096 x 14336, 1024, 107 and 93; 2048 x 4096 x 1024, 2048, 28 and
// 30; 2048 x 4096 x 4096, 2048, 47 and 61).
constexpr int64_t kSmallMost = 1024;

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_gemm_act(int64_t m, int64_t n, int64_t k, const uint8_t* a_codes, const uint8_t* a_scales,
                        const uint8_t* b_codes, const uint8_t* b_scales, const void* bias, fp4_dtype bias_type,
                        fp4_act act, const uint16_t* residual, int64_t ldr, uint16_t* z, void* y, fp4_dtype y_type,
                        int64_t ldy, hipStream_t stream) {
  if (!dtype_ok(bias_type) || !dtype_ok(y_type) || act < FP4_ACT_NONE || act > FP4_ACT_SILU) return FP4_EINVAL;
  if (m < 0 || !mult32z(n) || !mult32z(k) || k >= ((int64_t)1 << 24) || ldy < n || (residual && ldr < n)) return FP4_ESHAPE;
  if (m == 0 || n == 0) return FP4_OK;
  if (!y || (k > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return FP4_EINVAL;
  const int64_t tiles = tiles_of(m, BM, n, BN);
  if (tiles < 0) return FP4_ESHAPE;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(residual) ||
      !aligned16(z) || !aligned16(y) || (residual && ldr % 8 != 0) || ldy % (y_type == FP4_F32 ? 4 : 8) != 0 ||
      (reinterpret_cast<uintptr_t>(bias) & (bias_type == FP4_F32 ? 3 : 1)))
    return FP4_EALIGN;
  const bool f32 = y_type == FP4_F32;
  const Epilogue e{y, ldy, bias, residual, ldr, z, (int)act, f32, bias_type == FP4_F32, 0,
                   streams(m, n * ((f32 ? 4 : 2) + (z ? 2 : 0)))};
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, tile_grid(tiles), dim3(kFastThreads), 0, as_stream(stream), m, n, k, a_codes,
                       a_scales, b_codes, b_scales, e);
  };
  const int64_t small = tiles_of(m, kSmallTile, n, kSmallTile);
  if (small > 0 && small <= kSmallMost) {
    hipLaunchKernelGGL(gemm_act_small_kernel, dim3((unsigned)small), dim3(kSmallThreads), 0, as_stream(stream), m, n, k,
                       a_codes, a_scales, b_codes, b_scales, e);
    return launch_status();
  }
  const int mode = k_mode(k);
  if (mode == kWhole) go(gemm_act_kernel<kWhole>);
  else if (mode == kWindow) go(gemm_act_kernel<kWindow>);
  else go(gemm_act_kernel<kShort>);
  return launch_status();
}

}  // extern "C"
