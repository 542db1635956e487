// Few-row products of sorted tokens with their experts' weights
// (fp4_matvec_experts, fp4_swiglu_matvec_experts).
//
// A unit is a few rows of one expert's segment, sixteen at most; a row of workgroups
// takes one, and walks the expert's weights as the plain product does.  Which
// units there are is known on the device only: a launch has as many rows of
// workgroups as so many sorted rows can make, and the spare ones end at once.
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.2 (Eq. 1) decode,
// §2.4 row layouts, §3.2 gated FFN.
//
// Bound as the plain product: two of eight experts' gated 14336 x 4096, one row
// each (125 MB), 24 us, all eight (499 MB), two rows each, 103 us, 4.8 TB/s; 64
// experts' 2048 x 1056, three rows each (73 MB), 26 us, 19 without products behind
// the loads.  The CUs are shared out evenly among the experts, whatever the router
// does: of 64 experts' 192 rows, 129 on one expert and one on each other take 39 us, all
// on one 24 for 1 MB of weights.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "experts.h"
#include "matvec_core.h"

namespace mx {

struct ExpertRows {
  const int32_t* offsets;                                // [experts + 1]
  int experts, rows;
  int unit;                                              // rows of a unit, 16 at most
};

// First row, number of rows and expert of unit `unit`; false past the last.
__device__ __forceinline__ bool expert_unit(const ExpertRows& x, int unit, int& expert, int& first, int& count) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int at = 0; at < x.experts; at += 64) {
    const int e = at + lane;
    const int lo = std::min(std::max(x.offsets[std::min(e, x.experts)], 0), x.rows);
    const int hi = std::min(std::max(x.offsets[std::min(e + 1, x.experts)], lo), x.rows);
    const int mine = (int)((uint32_t)(hi - lo + x.unit - 1) / (uint32_t)x.unit);
    const int sum = wave_prefix_sum(mine);
    const uint64_t behind = __builtin_amdgcn_ballot_w64(unit < before + sum);
    if (behind) {
      const int src = __builtin_ctzll(behind);
      const int in = unit - before - __builtin_amdgcn_readlane(sum, src) + __builtin_amdgcn_readlane(mine, src);
      expert = at + src;
      first = __builtin_amdgcn_readlane(lo, src) + in * x.unit;
      count = std::min(__builtin_amdgcn_readlane(hi, src) - first, x.unit);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// Rows behind the last segment get 0 (few or none).
__device__ __forceinline__ void clear_behind(const ExpertRows& x, const MatvecArgs& a) {
  const int last = std::min(std::max(x.offsets[x.experts], 0), x.rows);
  const int64_t threads = (int64_t)gridDim.x * gridDim.y * blockDim.x;
  for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < (x.rows - last) * a.n; i += threads) {
    if (a.h) a.h[last * a.n + i] = 0;
    else a.c[(last + i / a.n) * a.ldc + i % a.n] = 0.0f;
  }
}

template <int XT, int U, bool GATE, bool STAGED, int SC>
__global__ __launch_bounds__(1024) void matvec_experts_kernel(MatvecArgs a, MvPlan plan, ExpertRows x) {
  clear_behind(x, a);
  int expert, first, count;
  if (!expert_unit(x, blockIdx.y, expert, first, count)) return;
  const int64_t n = GATE ? 2 * a.n : a.n;
  a.m = count;
  a.x = static_cast<const uint8_t*>(a.x) + first * (XT == kXBf16 ? 2 * a.ldx : a.ldx);
  a.x_scales += XT == kXBf16 ? 0 : first * (a.k >> 5);
  a.codes += expert * n * (a.k >> 1);
  a.scales += expert * n * (a.k >> 5);
  if (GATE) a.h += first * a.n;
  else a.c += first * a.ldc;
  matvec_body<XT, kMx, 1, 1, 16, U, GATE, STAGED, SC, false>(a, plan, MvEpilogue{});
}

// An empty reduction or one of a few weights an expert.
template <int XT, bool GATE>
__global__ __launch_bounds__(256) void matvec_experts_small_kernel(MatvecArgs a, ExpertRows x) {
  const uint8_t* const codes = a.codes;
  const uint8_t* const scales = a.scales;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < x.rows * a.n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / a.n, col = i % a.n;
    float v = 0.0f, w = 0.0f;
    int e = 0;
    while (a.k > 0 && e < x.experts && !(r >= x.offsets[e] && r < x.offsets[e + 1])) ++e;
    if (a.k > 0 && e < x.experts) {
      const int64_t weights = e * (GATE ? 2 : 1) * a.n * a.k;
      a.codes = codes + (weights >> 1);
      a.scales = scales + (weights >> 5);
      v = small_sum<XT>(a, r, col);
      if (GATE) w = small_sum<XT>(a, r, a.n + col);
    }
    if constexpr (GATE) {
      const uint32_t both = bf16_pack2_rne(v, w);
      const float av[1] = {__uint_as_float(both << 16)};
      float sig[1], sl[1];
      sigmoid_silu_n(av, sig, sl);
      a.h[i] = (uint16_t)bf16_pack2_rne(__fmul_rn(sl[0], __uint_as_float(both & 0xFFFF0000u)), 0.0f);
    } else {
      a.c[r * a.ldc + col] = v;
    }
  }
}

template <int XT, bool GATE>
static fp4_status matvec_experts_launch(MatvecArgs a, ExpertRows x, hipStream_t stream) {
  if ((GATE ? 2 : 1) * a.n * (a.k / 32) < 4) {
    const int64_t grid = std::min<int64_t>((x.rows * a.n + 255) / 256, 65536);
    hipLaunchKernelGGL((matvec_experts_small_kernel<XT, GATE>), dim3((unsigned)grid), dim3(256), 0, stream, a, x);
    return launch_status();
  }
  const int experts = std::min(x.experts, x.rows);       // that can have a row
  // Long rows of which LDS does not hold sixteen: units of as many as it holds, if
  // the experts have no more of them each, on average (8 experts' 4096 x 14336,
  // four rows each: 86 to 60 us, one to twelve: 100 to 85; the weights of an expert
  // with more are read again).
  const int64_t held = std::min<int64_t>(kStagedXBytes / stage_pitch(a.k), 16);
  x.unit = held > 0 && x.rows <= held * experts ? (int)held : 16;
  a.m = std::min(x.rows, x.unit);
  const int units = experts + x.rows / x.unit;           // a unit an expert, and one more for all its rows
  const int64_t cus = std::max<int64_t>(kMatvecGrid / experts, 1);
  matvec_variant<kMx, GATE, kWordScales, false>(a, cus, [&](auto v, const MvPlan& plan, unsigned grid) {
    using V = decltype(v);
    static_assert(V::MT == 1 && V::NT == 1 && V::NW == 16, "a unit is one tile of rows");
    hipLaunchKernelGGL((matvec_experts_kernel<XT, V::U, GATE, V::STAGED, V::SC>), dim3(grid, (unsigned)units), dim3(1024),
                       0, stream, a, plan, x);
  });
  return launch_status();
}

// Checks shared by the two calls.
static fp4_status experts_check(int64_t experts, int64_t rows, int64_t n, int64_t k, const int32_t* offsets, const void* x,
                                int64_t ldx, const uint8_t* x_scales, const uint8_t* codes, const uint8_t* scales,
                                const void* out) {
  if (!experts_ok(experts) || rows < 0 || rows > 65536) return FP4_ESHAPE;
  const fp4_status st = matvec_check(std::min<int64_t>(rows, 1), n, k, x, ldx, x_scales, x_scales != nullptr, codes, scales, out);
  if (st != FP4_OK || rows == 0 || n == 0) return st;
  if (!offsets) return FP4_EINVAL;
  return (reinterpret_cast<uintptr_t>(offsets) & 3) ? FP4_EALIGN : FP4_OK;
}

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_matvec_experts(int64_t experts, int64_t rows, int64_t n, int64_t k, const int32_t* offsets, const void* x,
                              int64_t ldx, const uint8_t* x_scales, const uint8_t* w_codes, const uint8_t* w_scales, float* c,
                              int64_t ldc, hipStream_t stream) {
  if (ldc < n || (x_scales && ldx != k)) return FP4_ESHAPE;
  const fp4_status st = experts_check(experts, rows, n, k, offsets, x, ldx, x_scales, w_codes, w_scales, c);
  if (st != FP4_OK || rows == 0 || n == 0) return st;
  if (reinterpret_cast<uintptr_t>(c) & 3) return FP4_EALIGN;
  const MatvecArgs a{0, n, k, x, ldx, x_scales, w_codes, w_scales, nullptr, 0, c, ldc, 0, nullptr};
  const ExpertRows r{offsets, (int)experts, (int)rows, 0};
  return x_scales ? matvec_experts_launch<kXE4m3, false>(a, r, as_stream(stream))
                  : matvec_experts_launch<kXBf16, false>(a, r, as_stream(stream));
}

fp4_status fp4_swiglu_matvec_experts(int64_t experts, int64_t rows, int64_t f, int64_t d, const int32_t* offsets,
                                     const void* x, int64_t ldx, const uint8_t* x_scales, const uint8_t* w13_codes,
                                     const uint8_t* w13_scales, uint16_t* h, hipStream_t stream) {
  if (x_scales && ldx != d) return FP4_ESHAPE;
  const fp4_status st = experts_check(experts, rows, f, d, offsets, x, ldx, x_scales, w13_codes, w13_scales, h);
  if (st != FP4_OK || rows == 0 || f == 0) return st;
  if (reinterpret_cast<uintptr_t>(h) & 1) return FP4_EALIGN;
  const MatvecArgs a{0, f, d, x, ldx, x_scales, w13_codes, w13_scales, nullptr, 0, nullptr, 0, 0, h};
  const ExpertRows r{offsets, (int)experts, (int)rows, 0};
  return x_scales ? matvec_experts_launch<kXE4m3, true>(a, r, as_stream(stream))
                  : matvec_experts_launch<kXBf16, true>(a, r, as_stream(stream));
}

}  // extern "C"
