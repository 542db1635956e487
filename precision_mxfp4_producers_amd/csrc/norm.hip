// The boundary before a quantized linear layer: dropout of the incoming
// branch, its addition to the residual stream, RMSNorm, and the norm's output
// as E4M3 or E2M1 codes with E8M0 scales (fp4_rmsnorm_producer), the gradients
// of that boundary (fp4_rmsnorm_backward), and dropout alone (fp4_dropout).
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §3.1-§3.2 (a
// producer completes every scale group its consumer reads and keeps the bf16
// residual and the row statistics); §2.2.1 upward scales.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "dropout.h"
#include "rows.h"

namespace mx {

// ---------------------------------------------------------------- dropout
// out = bf16(dropout(x) [+ residual]); one thread per group of eight columns.
// Bound by HBM: bf16 8192 x 14336, 470 MB, takes 80-84 us (5.6-5.9 TB/s; a 1 GiB
// copy moves 5.2); the generator is some 400 of a wave's cycles per 3 KB.  With
// a residual it is not: that it may be absent is known at run time only, which
// keeps its values in scratch memory (fp32 x, 940 MB: 246 us, 3.8 TB/s).
// VEC: every row of every tensor starts on a 16-byte boundary; a group that
// runs past the row's end, and every group otherwise, goes element by element
// (a view's last row may end with its last element).
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(int64_t groups, uint32_t per, int64_t cols, const void* x,
                                                      int64_t ldx, const uint16_t* residual, int64_t ldr,
                                                      uint16_t* out, int64_t ldo, Dropout d) {
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < groups; q += (int64_t)gridDim.x * 256) {
    const int64_t r = groups <= 0xFFFFFFFF ? (int64_t)((uint32_t)q / per) : q / per;
    const int64_t c = (q - r * per) * 8;
    float v[8], base[8];
    const bool whole = VEC && c + 8 <= cols;
    if (whole) {
      load8<F32>(x, r * ldx + c, v);
      if (residual) unpack8(load_once_u4(residual + r * ldr + c), base);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = base[j] = 0.0f;
        if (c + j < cols) {
          v[j] = load1<F32>(x, r * ldx + c + j);
          if (residual) base[j] = bf16_bits_to_f32(residual[r * ldr + c + j]);
        }
      }
    }
    dropout8(v, residual ? base : nullptr, (uint64_t)q, d);
    if (whole) {
      *reinterpret_cast<uint4*>(out + r * ldo + c) = pack8(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) out[r * ldo + c + j] = (uint16_t)f32_to_bf16_rne(v[j]);
    }
  }
}

// ---------------------------------------------------------------- RMSNorm producer
// Sum over the G threads of a row (G a power of two, 16 <= G <= 1024): lanes
// of a wave by exchanges, waves of a workgroup through LDS in wave order.  The
// same value in every thread of the row.
template <int G, typename T>
__device__ __forceinline__ T row_sum(T v, T* lds) {
#pragma unroll
  for (int s = 1; s < (G < 64 ? G : 64); s <<= 1) v = v + __shfl_xor(v, s, 64);
  if constexpr (G > 64) {
    __syncthreads();                                     // the previous use of lds is over
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < G / 64; ++w) v = v + lds[w];
  }
  return v;
}

constexpr int kNoRemainder = 0x267;                      // the classes of both zeros, both infinities and NaN

// A launch's dimension holds less than 2^32 threads (a larger one wraps, with
// no error), fewer than the calls take rows of (17 GB of bf16 at 32 columns):
// workgroups past 2^20 go to a second dimension, in equal shares.  A return of
// the few past the last row, in place of their clamped loads, cost every launch
// of 1536 to 2048 columns 2-3%.
constexpr int64_t kNormGridX = 1 << 20;

struct NormOut {
  uint16_t* sum;                                         // any of these may be null
  uint16_t* y;
  float* rstd;
  uint8_t* codes;
  uint8_t* scales;
  int e4m3;                                              // format of the codes
};

// s = bf16(dropout(x) + residual); rstd = 1 / sqrt(mean(s^2) + eps);
// y = bf16((s rstd) gamma), then codes and scales of y.  The norm is taken of
// the rounded s, the tensor that the backward pass and the next boundary read,
// and the codes of the rounded y, so that they are the bytes that a separate
// quantizer call on y gives (row and column views of one y agree).
// G threads hold one row, thread i the groups of eight columns i, i + G, ...:
// the row stays in registers between the statistics and the output, x and the
// residual are read once.  Four neighbouring lanes hold one 32-value block.
//
// The sum may take the residual's place: a thread that stores it has read those
// elements, and uses no others (what it reads past the end is dropped).
//
// No branch surrounds a load (a row or column past the end reads the last
// one), and all of a thread's loads go out before its first use: 8192 x 4096,
// fp32 x with dropout and residual to s and E4M3, 302 MB, takes 52 us (5.8
// TB/s), and took 89 with the loads of each group of columns behind the stores
// of the one before.  Bound by HBM; one token by its launch (3.3 us).
template <int G, int V, bool F32, bool RES>
__global__ __launch_bounds__(G < 256 ? 256 : G) void rmsnorm_kernel(int64_t t, int d, const void* __restrict__ x,
                                                                    int64_t ldx, const uint16_t* residual,
                                                                    int64_t ldr, const uint16_t* __restrict__ gamma,
                                                                    float eps, double inv_d, Dropout drop, NormOut o) {
  constexpr int kRows = G < 256 ? 256 / G : 1;
  __shared__ double lds[16];
  const int i = threadIdx.x & (G - 1);
  const int64_t r = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows + (G < 256 ? threadIdx.x / G : 0);
  const int64_t rr = std::min(r, t - 1);
  uint4 s[V], g[V];
  float v[V][8], base[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = std::min((k * G + i) * 8, d - 8);
    load8<F32>(x, rr * ldx + c, v[k]);
    if constexpr (RES) unpack8(load_once_u4(residual + rr * ldr + c), base[k]);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) g[k] = *reinterpret_cast<const uint4*>(gamma + std::min((k * G + i) * 8, d - 8));
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * G + i) * 8;
    const bool live = r < t && c < d;                    // whole rows of threads, and whole groups of four lanes
    if (drop.thr) {
      dropout8(v[k], RES ? base[k] : nullptr, (uint64_t)rr * (uint32_t)(d >> 3) + (uint32_t)(c >> 3), drop);
    } else if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = __fadd_rn(v[k][j], base[k][j]);
    }
    s[k] = pack8(v[k]);
    if (!live) s[k] = make_uint4(0, 0, 0, 0);
    if (o.sum && live) *reinterpret_cast<uint4*>(o.sum + r * d + c) = s[k];
    unpack8(s[k], v[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[k][j], v[k][j], sq);
  }
  // The statistic in 64 bits from the threads' sums on: one Newton step from
  // the fp32 root, then as a pair rstd + low.
  const double mean = __builtin_fma(row_sum<G>((double)sq, lds), inv_d, (double)eps);
  double r64 = (double)__fdiv_rn(1.0f, __fsqrt_rn((float)mean));
  r64 = r64 * __builtin_fma(-0.5 * mean * r64, r64, 1.5);
  const float rstd = (float)r64, low = (float)(r64 - (double)rstd);
  if (r < t && i == 0) o.rstd[r] = rstd;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * G + i) * 8;
    const bool live = r < t && c < d;
    float w[8], gm[8];
    unpack8(s[k], w);
    unpack8(g[k], gm);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // s (rstd + low) gamma with the products' remainders: what bf16 and the
      // codes round is off by one fp32 rounding, not by that of three steps.
      // A zero keeps its sign, and a product past fp32 its infinity, of which
      // the remainder would make a NaN.
      const float a = __fmul_rn(w[j], rstd), ar = __builtin_fmaf(w[j], low, __builtin_fmaf(w[j], rstd, -a));
      const float b = __fmul_rn(a, gm[j]);
      const float sum = __fadd_rn(b, __builtin_fmaf(ar, gm[j], __builtin_fmaf(a, gm[j], -b)));
      w[j] = __builtin_amdgcn_classf(b, kNoRemainder) ? b : sum;
    }
    const uint4 y = pack8(w);
    if (o.y && live) *reinterpret_cast<uint4*>(o.y + r * d + c) = y;
    if (o.codes) {
      const uint32_t am = max_quad(bf16_absmax8(y.x, y.y, y.z, y.w)) << 16;
      const int e = o.e4m3 ? upward_exp_e4m3(am) : upward_exp(am);
      if (live) {
        if (o.e4m3)
          *reinterpret_cast<uint2*>(o.codes + r * d + c) = e4m3_8(y, pow2_scale(e));
        else
          *reinterpret_cast<uint32_t*>(o.codes + ((r * d + c) >> 1)) = rtn8_bf16(y.x, y.y, y.z, y.w, pow2_scale(e));
        if ((i & 3) == 0) o.scales[(r * d + c) >> 5] = (uint8_t)(e + 127);
      }
    }
  }
}

// ---------------------------------------------------------------- RMSNorm backward
// With xh = s rstd and g = dy gamma,
//   ds' = rstd (g - xh mean(g xh)) [+ ds],  dsum = bf16(ds'),
//   dx = bf16(dropout(ds')),  dgamma = sum over rows of dy xh.
// G threads hold a row, as in the forward.  A workgroup walks rows in steps of
// the whole grid, loads the next row's tensors before it works on the current
// one, keeps its columns' share of dgamma in registers and writes it once, as
// one row of the workspace.  Bound by HBM: fp32 dy 8192 x 4096 with ds and
// dropout, 403 MB, takes 70 us and 5 for the sums of dgamma (88 and 10 without
// the next row's loads and with one column a thread in the sums).
template <int V, bool F32, bool DS>
struct BwdRow {
  float dy[V][8];
  uint4 s[V], ds[V];
  float rstd;
};

template <int G, int V, bool F32, bool DS>
__global__ __launch_bounds__(G < 256 ? 256 : G) void rmsnorm_bwd_kernel(
    int64_t t, int d, const void* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ s, int64_t lds_s,
    const float* __restrict__ rstd, const uint16_t* __restrict__ gamma, const uint16_t* __restrict__ ds, int64_t ldds,
    Dropout drop, uint16_t* __restrict__ dsum, uint16_t* __restrict__ dx, float* __restrict__ parts) {
  constexpr int kRows = G < 256 ? 256 / G : 1;
  constexpr bool NEXT = G < 512;                         // the next row's registers beside this one's
  __shared__ float lds[G < 256 ? 4 * 64 * V * 8 : 16];
  const int i = threadIdx.x & (G - 1);
  const int64_t first = (int64_t)blockIdx.x * kRows + (G < 256 ? threadIdx.x / G : 0), sweep = (int64_t)gridDim.x * kRows;
  const int64_t turns = (t - (int64_t)blockIdx.x * kRows + sweep - 1) / sweep;   // the same for a whole workgroup
  float dg[V][8];
  uint4 gm[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    gm[k] = *reinterpret_cast<const uint4*>(gamma + std::min((k * G + i) * 8, d - 8));
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[k][j] = 0.0f;
  }
  const auto load = [&](BwdRow<V, F32, DS>& row, int64_t turn) {
    const int64_t r = std::min(first + turn * sweep, t - 1);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = std::min((k * G + i) * 8, d - 8);
      load8<F32>(dy, r * lddy + c, row.dy[k]);
      row.s[k] = load_once_u4(s + r * lds_s + c);
      if constexpr (DS) row.ds[k] = load_once_u4(ds + r * ldds + c);
    }
    row.rstd = rstd[r];
  };
  BwdRow<V, F32, DS> cur, next;
  load(cur, 0);
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t r = first + turn * sweep;
    if constexpr (NEXT) load(next, turn + 1);
    float dot = 0.0f;
    const float rs = cur.rstd;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const bool live = r < t && (k * G + i) * 8 < d;
      float xh[8], g[8];
      unpack8(cur.s[k], xh);
      unpack8(gm[k], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!live) cur.dy[k][j] = 0.0f;
        xh[j] = __fmul_rn(xh[j], rs);
        // selected, not multiplied by 0: a dead lane holds the last row's s, which may be an infinity
        dg[k][j] = live ? __builtin_fmaf(cur.dy[k][j], xh[j], dg[k][j]) : dg[k][j];
        dot = live ? __builtin_fmaf(__fmul_rn(cur.dy[k][j], g[j]), xh[j], dot) : dot;
      }
    }
    const float mean = __fdiv_rn(row_sum<G>(dot, lds), (float)d);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * G + i) * 8;
      if (r < t && c < d) {
        float v[8], xh[8], g[8], b[8];
        unpack8(cur.s[k], xh);
        unpack8(gm[k], g);
        if constexpr (DS) unpack8(cur.ds[k], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = __builtin_fmaf(-__fmul_rn(xh[j], rs), mean, __fmul_rn(cur.dy[k][j], g[j]));
          v[j] = DS ? __builtin_fmaf(rs, v[j], b[j]) : __fmul_rn(rs, v[j]);
        }
        *reinterpret_cast<uint4*>(dsum + r * d + c) = pack8(v);
        if (drop.thr) {
          dropout8(v, nullptr, (uint64_t)r * (uint32_t)(d >> 3) + (uint32_t)(c >> 3), drop);
          *reinterpret_cast<uint4*>(dx + r * d + c) = pack8(v);
        }
      }
    }
    if constexpr (NEXT) cur = next;
    else if (turn + 1 < turns) load(cur, turn + 1);
  }
  float* const out = parts + (int64_t)blockIdx.x * d;
  if constexpr (G < 256) {
    // lanes that hold the same columns of other rows, then the four waves
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int st = G; st < 64; st <<= 1) dg[k][j] = __fadd_rn(dg[k][j], __shfl_xor(dg[k][j], st, 64));
        lds[(((threadIdx.x >> 6) * V + k) * 8 + j) * 64 + (threadIdx.x & 63)] = dg[k][j];
      }
    __syncthreads();
    for (int e = threadIdx.x; e < V * G * 8; e += 256) {
      const int l = e & (G - 1), j = (e / G) & 7, k = e / (G * 8), c = (k * G + l) * 8 + j;
      if (c >= d) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v = __fadd_rn(v, lds[((w * V + k) * 8 + j) * 64 + l]);
      out[c] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * G + i) * 8;
      if (c < d) {
        float4* const p = reinterpret_cast<float4*>(out + c);
        p[0] = make_float4(dg[k][0], dg[k][1], dg[k][2], dg[k][3]);
        p[1] = make_float4(dg[k][4], dg[k][5], dg[k][6], dg[k][7]);
      }
    }
  }
}

// dgamma[c] (+)= sum over the workspace's rows, in a fixed order: 32 slices of
// rows per column, added by slice.  32 columns (one 128-byte line a row) a
// workgroup, four a thread, so that a thread's loads are wide and few.
__global__ __launch_bounds__(256) void dgamma_kernel(int64_t rows, int d, const float* __restrict__ parts,
                                                     float* __restrict__ dgamma, int accumulate) {
  __shared__ float4 lds[32][9];
  const int cl = threadIdx.x & 7, sl = threadIdx.x >> 3, c = blockIdx.x * 32 + cl * 4;   // d is a multiple of 32
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int64_t q = sl; q < rows; q += 32) {
    const float4 p = *reinterpret_cast<const float4*>(parts + q * d + c);
    v = make_float4(__fadd_rn(v.x, p.x), __fadd_rn(v.y, p.y), __fadd_rn(v.z, p.z), __fadd_rn(v.w, p.w));
  }
  lds[sl][cl] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int col = blockIdx.x * 32 + threadIdx.x;
    const float* const f = reinterpret_cast<const float*>(lds);
    float sum = accumulate ? dgamma[col] : 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) sum = __fadd_rn(sum, f[q * 36 + threadIdx.x]);
    dgamma[col] = sum;
  }
}

// ---------------------------------------------------------------- host side
constexpr int64_t kNormMaxD = 32768;                     // a row in the registers of 1024 threads, 32 values each
// Calls f with the variant that holds a row of d columns: threads a row, groups of eight columns a thread.
template <typename F>
static void norm_variant(int64_t d, F&& f) {
  using std::integral_constant;
#define MX_NORM(G, V) f(integral_constant<int, G>{}, integral_constant<int, V>{})
  if (d <= 128) MX_NORM(16, 1);
  else if (d <= 512) MX_NORM(64, 1);
  else if (d <= 1024) MX_NORM(64, 2);
  else if (d <= 1536) MX_NORM(64, 3);
  else if (d <= 2048) MX_NORM(64, 4);
  else if (d <= 4096) MX_NORM(256, 2);
  else if (d <= 6144) MX_NORM(256, 3);
  else if (d <= 8192) MX_NORM(256, 4);
  else if (d <= 16384) MX_NORM(512, 4);
  else MX_NORM(1024, 4);
#undef MX_NORM
}

// Workgroups of the backward pass, each of which leaves one row of partial
// sums: two a CU where that gives each several rows, else one a CU at most (a
// row of sums costs as much to write and read back as two rows of inputs).
static int64_t norm_parts(int64_t t, int64_t d) {
  const int64_t rows = d <= 128 ? 16 : d <= 2048 ? 4 : 1, groups = t / rows + (t % rows != 0);
  return groups >= 2048 ? 512 : std::min<int64_t>(groups, 256);
}

static bool prob_ok(float p) { return p >= 0.0f && p <= 1.0f; }             // false for NaN
static bool pitch_ok(fp4_dtype t, int64_t ld) { return ld % (t == FP4_F32 ? 4 : 8) == 0; }

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_dropout(int64_t rows, int64_t cols, const void* x, fp4_dtype x_type, int64_t ldx,
                       const uint16_t* residual, int64_t ldr, float p, uint64_t seed, uint64_t offset, uint16_t* out,
                       int64_t ldo, hipStream_t stream) {
  if (!dtype_ok(x_type) || !prob_ok(p)) return FP4_EINVAL;
  if (rows < 0 || cols < 0 || ldx < cols || ldo < cols || (residual && ldr < cols)) return FP4_ESHAPE;
  if (rows == 0 || cols == 0) return FP4_OK;
  if (!x || !out) return FP4_EINVAL;
  const int64_t per = (cols - 1) / 8 + 1;
  if (per > 0x7FFFFFFF || rows > ((int64_t)1 << 56) / per) return FP4_ESHAPE;
  const uintptr_t low = x_type == FP4_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(x) & low) || (reinterpret_cast<uintptr_t>(residual) & 1) ||
      (reinterpret_cast<uintptr_t>(out) & 1))
    return FP4_EALIGN;
  const bool vec = aligned16(x) && aligned16(residual) && aligned16(out) && pitch_ok(x_type, ldx) && ldo % 8 == 0 &&
                   (!residual || ldr % 8 == 0);
  const int64_t groups = rows * per;
  const unsigned grid = (unsigned)std::min<int64_t>((groups + 255) / 256, 1 << 20);
  const Dropout d = make_dropout(p, seed, offset);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, as_stream(stream), groups, (uint32_t)per, cols, x, ldx,
                       residual, ldr, out, ldo, d);
  };
  if (x_type == FP4_F32) vec ? go(dropout_kernel<true, true>) : go(dropout_kernel<true, false>);
  else vec ? go(dropout_kernel<false, true>) : go(dropout_kernel<false, false>);
  return launch_status();
}

fp4_status fp4_rmsnorm_producer(int64_t t, int64_t d, const void* x, fp4_dtype x_type, int64_t ldx,
                                const uint16_t* residual, int64_t ldr, const uint16_t* gamma, float eps, float p,
                                uint64_t seed, uint64_t offset, uint16_t* sum, float* rstd, uint16_t* y,
                                fp4_format format, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (!dtype_ok(x_type) || !prob_ok(p) || (format != FP4_E2M1 && format != FP4_E4M3)) return FP4_EINVAL;
  if (!(eps > 0.0f) || !(eps <= 3.4028234e38f) || (codes == nullptr) != (scales == nullptr)) return FP4_EINVAL;
  if (t < 0 || !mult32z(d) || d > kNormMaxD || ldx < d || (residual && ldr < d)) return FP4_ESHAPE;
  if (t == 0 || d == 0) return FP4_OK;
  if (t > 0x7FFFFFFF) return FP4_ESHAPE;
  if (!x || !gamma || !rstd) return FP4_EINVAL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(sum) || !aligned16(y) ||
      !aligned16(codes) || (reinterpret_cast<uintptr_t>(rstd) & 3) || !pitch_ok(x_type, ldx) ||
      (residual && ldr % 8 != 0))
    return FP4_EALIGN;
  const Dropout drop = make_dropout(p, seed, offset);
  const NormOut o{sum, y, rstd, codes, scales, format == FP4_E4M3};
  norm_variant(d, [&](auto g, auto v) {
    constexpr int G = g(), V = v(), kRows = G < 256 ? 256 / G : 1;
    const int64_t groups = (t + kRows - 1) / kRows, shares = (groups + kNormGridX - 1) / kNormGridX;
    const dim3 grid((unsigned)((groups + shares - 1) / shares), (unsigned)shares);
    const auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(G < 256 ? 256 : G), 0, as_stream(stream), t, (int)d, x, ldx,
                         residual, ldr, gamma, eps, 1.0 / (double)d, drop, o);
    };
    if (residual) x_type == FP4_F32 ? go(rmsnorm_kernel<G, V, true, true>) : go(rmsnorm_kernel<G, V, false, true>);
    else x_type == FP4_F32 ? go(rmsnorm_kernel<G, V, true, false>) : go(rmsnorm_kernel<G, V, false, false>);
  });
  return launch_status();
}

int64_t fp4_rmsnorm_backward_workspace(int64_t t, int64_t d) {
  if (t < 0 || !mult32z(d) || d > kNormMaxD) return -1;
  return norm_parts(t, d) * d * (int64_t)sizeof(float);
}

fp4_status fp4_rmsnorm_backward(int64_t t, int64_t d, const void* dy, fp4_dtype dy_type, int64_t lddy,
                                const uint16_t* s, int64_t lds, const float* rstd, const uint16_t* gamma,
                                const uint16_t* ds, int64_t ldds, float p, uint64_t seed, uint64_t offset,
                                uint16_t* dsum, uint16_t* dx, float* dgamma, int accumulate, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dy_type) || !prob_ok(p) || (accumulate != 0 && accumulate != 1)) return FP4_EINVAL;
  if (t < 0 || !mult32z(d) || d > kNormMaxD || lddy < d || lds < d || (ds && ldds < d)) return FP4_ESHAPE;
  if (d == 0) return FP4_OK;
  if (t > 0x7FFFFFFF) return FP4_ESHAPE;
  if (!dgamma) return FP4_EINVAL;
  const Dropout drop = make_dropout(p, seed, offset);
  if (t > 0 && (!dy || !s || !rstd || !gamma || !dsum || (drop.thr && !dx) || !workspace)) return FP4_EINVAL;
  if (workspace_bytes < fp4_rmsnorm_backward_workspace(t, d)) return FP4_ESHAPE;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(gamma) || !aligned16(ds) || !aligned16(dsum) || !aligned16(dx) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(rstd) & 3) || (reinterpret_cast<uintptr_t>(dgamma) & 3) ||
      !pitch_ok(dy_type, lddy) || lds % 8 != 0 || (ds && ldds % 8 != 0))
    return FP4_EALIGN;
  const int64_t rows = norm_parts(t, d);
  float* parts = static_cast<float*>(workspace);
  if (t > 0)
    norm_variant(d, [&](auto g, auto v) {
      constexpr int G = g(), V = v();
      const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)rows), dim3(G < 256 ? 256 : G), 0, as_stream(stream), t, (int)d, dy,
                           lddy, s, lds, rstd, gamma, ds, ldds, drop, dsum, dx, parts);
      };
      if (ds) dy_type == FP4_F32 ? go(rmsnorm_bwd_kernel<G, V, true, true>) : go(rmsnorm_bwd_kernel<G, V, false, true>);
      else dy_type == FP4_F32 ? go(rmsnorm_bwd_kernel<G, V, true, false>) : go(rmsnorm_bwd_kernel<G, V, false, false>);
    });
  hipLaunchKernelGGL(dgamma_kernel, dim3((unsigned)(d / 32)), dim3(256), 0, as_stream(stream), rows, (int)d, parts,
                     dgamma, accumulate);
  return launch_status();
}

}  // extern "C"
