// Gradients of the products' epilogue (fp4_act_backward): dz = dy act'(z) and
// the bias' gradient, the column sums of dy act'(z).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "activation.h"
#include "rows.h"

namespace mx {

struct ActGradArgs {
  const void* dy;                                        // [m][lddy] bf16 or fp32
  int64_t lddy;
  const uint16_t* z;                                     // [m][ldz]
  int64_t ldz;
  uint16_t* dz;                                          // [m][n]
  float* sums;                                           // [row groups][n], or dbias, or null
  int64_t m, n;
  int64_t rows;                                          // rows of a workgroup
  int accumulate;                                        // sums is dbias and keeps what it holds
  int stream;                                            // dz past the caches
};

// A workgroup takes 8 << LG columns (eight a thread) of `rows` rows; the 256 >>
// LG threads of a column group take every so many rows, and their sums meet in
// LDS in order: deterministic.  Bound by memory: 8192 x 14336 with fp32 dy,
// 940 MB, take 179 us, 5.2 TB/s as a copy does, and the partial sums 4.9.
template <int ACT, bool F32, int LG>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  constexpr int L = 256 >> LG;
  __shared__ float lds[256 * 8];
  const int lane = threadIdx.x & ((1 << LG) - 1), rl = threadIdx.x >> LG;
  const int64_t c = ((int64_t)blockIdx.x << (LG + 3)) + lane * 8;
  const int64_t first = (int64_t)blockIdx.y * a.rows, last = std::min(first + a.rows, a.m);
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.n) {
    for (int64_t r = first + rl; r < last; r += L) {
      float y[8], z[8];
      load8<F32>(a.dy, r * a.lddy + c, y);
      unpack8(load_once_u4(a.z + r * a.ldz + c), z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = __fmul_rn(y[j], act_slope<ACT>(z[j]));
        sum[j] = __fadd_rn(sum[j], y[j]);
      }
      put(reinterpret_cast<u32x4v*>(a.dz + r * a.n + c), __builtin_bit_cast(u32x4v, pack8(y)), a.stream);
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) lds[j * 256 + threadIdx.x] = sum[j];
  __syncthreads();
  for (int q = threadIdx.x; q < 8 << LG; q += 256) {
    const int64_t col = ((int64_t)blockIdx.x << (LG + 3)) + q;
    if (col >= a.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < L; ++w) v = __fadd_rn(v, lds[(q & 7) * 256 + (w << LG) + (q >> 3)]);
    float* const p = a.sums + blockIdx.y * a.n + col;
    *p = a.accumulate ? __fadd_rn(*p, v) : v;
  }
}

// dbias[c] (+)= the sum of the row groups' sums, in a fixed order: 32 slices of
// them a column, added by slice.  32 columns (one 128-byte line a row) a
// workgroup, four a thread.
__global__ __launch_bounds__(256) void act_grad_sum_kernel(int64_t groups, int64_t n, const float* __restrict__ sums,
                                                           float* __restrict__ dbias, int accumulate) {
  __shared__ float4 lds[32][9];
  const int cl = threadIdx.x & 7, sl = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl * 4;   // n is a multiple of 32
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int64_t q = sl; q < groups; q += 32) {
    const float4 p = *reinterpret_cast<const float4*>(sums + q * n + c);
    v = make_float4(__fadd_rn(v.x, p.x), __fadd_rn(v.y, p.y), __fadd_rn(v.z, p.z), __fadd_rn(v.w, p.w));
  }
  lds[sl][cl] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const float* const f = reinterpret_cast<const float*>(lds);
    float sum = accumulate ? dbias[col] : 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) sum = __fadd_rn(sum, f[q * 36 + threadIdx.x]);
    dbias[col] = sum;
  }
}

// dbias of no rows.
__global__ __launch_bounds__(256) void act_grad_zero_kernel(int64_t n, float* dbias) {
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < n; c += (int64_t)gridDim.x * 256) dbias[c] = 0.0f;
}

struct ActPlan {
  int lg;
  int64_t strips, groups, rows;                          // workgroups across columns and rows, rows of each
};

// Eight workgroups a CU where there are rows for that, each of several turns (a
// turn is 256 >> lg rows); one group of rows, whose sums are dbias at once, where
// that leaves it four turns at most.
static ActPlan act_plan(int64_t m, int64_t n) {
  const int lg = n > 128 ? 5 : (n > 64 ? 4 : (n > 32 ? 3 : 2));
  const int64_t strips = (n + (8 << lg) - 1) / (8 << lg), turn = 256 >> lg, turns = (m + turn - 1) / turn;
  const int64_t groups = std::max<int64_t>(std::min({(2048 + strips - 1) / strips, (turns + 3) / 4, (int64_t)512}), 1);
  const int64_t rows = (turns + groups - 1) / groups * turn;
  return ActPlan{lg, strips, std::max<int64_t>((m + rows - 1) / std::max<int64_t>(rows, 1), 1), rows};
}

template <int ACT>
static void act_grad_launch(const ActGradArgs& a, const ActPlan& p, bool f32, hipStream_t s) {
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.strips, (unsigned)p.groups), dim3(256), 0, s, a);
  };
  const auto by = [&](auto lg) { f32 ? go(act_grad_kernel<ACT, true, lg()>) : go(act_grad_kernel<ACT, false, lg()>); };
  if (p.lg == 5) by(std::integral_constant<int, 5>{});
  else if (p.lg == 4) by(std::integral_constant<int, 4>{});
  else if (p.lg == 3) by(std::integral_constant<int, 3>{});
  else by(std::integral_constant<int, 2>{});
}

static bool act_shape_ok(int64_t m, int64_t n) {
  return m >= 0 && m <= ((int64_t)1 << 40) && mult32z(n) && n <= ((int64_t)1 << 28);
}

}  // namespace mx

using namespace mx;

extern "C" {

int64_t fp4_act_backward_workspace(int64_t m, int64_t n) {
  if (!act_shape_ok(m, n)) return -1;
  if (m == 0 || n == 0) return 0;
  const ActPlan p = act_plan(m, n);
  return p.groups > 1 ? p.groups * n * (int64_t)sizeof(float) : 0;
}

fp4_status fp4_act_backward(int64_t m, int64_t n, const void* dy, fp4_dtype dy_type, int64_t lddy, const uint16_t* z,
                            int64_t ldz, fp4_act act, uint16_t* dz, float* dbias, int accumulate, void* workspace,
                            int64_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_type) || act < FP4_ACT_NONE || act > FP4_ACT_SILU || (accumulate != 0 && accumulate != 1)) return FP4_EINVAL;
  if (!act_shape_ok(m, n) || lddy < n || ldz < n) return FP4_ESHAPE;
  if (n == 0 || (m == 0 && (!dbias || accumulate))) return FP4_OK;
  if (m > 0 && (!dy || !z || !dz)) return FP4_EINVAL;
  if (!aligned16(dy) || !aligned16(z) || !aligned16(dz) || (reinterpret_cast<uintptr_t>(dbias) & 3) || !aligned16(workspace) ||
      lddy % (dy_type == FP4_F32 ? 4 : 8) != 0 || ldz % 8 != 0)
    return FP4_EALIGN;
  if (m == 0) {
    hipLaunchKernelGGL(act_grad_zero_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0,
                       as_stream(stream), n, dbias);
    return launch_status();
  }
  const ActPlan p = act_plan(m, n);
  const bool partial = dbias && p.groups > 1;
  if (partial && workspace_bytes < fp4_act_backward_workspace(m, n)) return FP4_ESHAPE;
  if (partial && !workspace) return FP4_EINVAL;
  const ActGradArgs a{dy, lddy, z, ldz, dz, partial ? static_cast<float*>(workspace) : dbias, m, n, p.rows,
                      partial ? 0 : accumulate, streams(m, n * 2)};
  const bool f32 = dy_type == FP4_F32;
  hipStream_t s = as_stream(stream);
  switch (act) {
    case FP4_ACT_RELU: act_grad_launch<FP4_ACT_RELU>(a, p, f32, s); break;
    case FP4_ACT_GELU: act_grad_launch<FP4_ACT_GELU>(a, p, f32, s); break;
    case FP4_ACT_GELU_TANH: act_grad_launch<FP4_ACT_GELU_TANH>(a, p, f32, s); break;
    case FP4_ACT_SILU: act_grad_launch<FP4_ACT_SILU>(a, p, f32, s); break;
    default: act_grad_launch<FP4_ACT_NONE>(a, p, f32, s);
  }
  const fp4_status st = launch_status();
  if (st != FP4_OK || !partial) return st;
  hipLaunchKernelGGL(act_grad_sum_kernel, dim3((unsigned)(n / 32)), dim3(256), 0, s, p.groups, n,
                     static_cast<const float*>(workspace), dbias, accumulate);
  return launch_status();
}

}  // extern "C"
