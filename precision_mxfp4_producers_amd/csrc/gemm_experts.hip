// Block-scaled E2M1 products of sorted tokens with their experts' weights
// (fp4_gemm_experts), the weights' gradients (fp4_gemm_experts_wgrad) and the
// gated FFN's producer per expert (fp4_swiglu_producer_experts), on the fast
// main loop and the epilogues of the plain products.
//
// Where the experts' segments lie is known on the device only: a launch has the
// tiles that its rows can need at most, and every workgroup finds its tile from
// the segment offsets (128 of them a turn, two a lane; under 1 us).
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.3 (Eq. 4-6) the
// contractions, §3.2 the gated FFN.
//
// Bound by the matrix cores, the tiles' start and end that short K leaves bare,
// and the weight gradients' stores.  Medians, operands from memory: 64 experts of 2048 x
// 2048, 65536 rows of a router that likes some experts better: rows 218 us (0.55 TFLOP,
// 2.5 PFLOP/s; a segment's last tile is half empty on average, 13% of them all), weight
// gradients 353 us (1.07 GB of fp32 at 3.1 TB/s; a fill of as much takes 158), the gated
// producer 583 (1.1 TFLOP, 1.9 PFLOP/s: its epilogue of three passes, and 830 MB
// written).  Few rows and few tiles take tiles of 64 x 64, but for the gated producer: 64
// experts' 2048 x 2048 with eight rows each, 285 MB, take it 139 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "experts.h"
#include "gemm_core.h"
#include "gemm_epilogue.h"
#include "gemm_small.h"
#include "swiglu_epilogue.h"

namespace mx {

// One output tile of a product over sorted rows.
struct ExpertTile {
  int expert;                                            // the number of experts: the rows behind the last segment
  int m0, end;                                           // first row, end of the segment
  int tn;                                                // column tile
};

// The tile of workgroup `pid`; false where there is none.  Tiles are counted
// expert by expert, the rows behind the last segment as one more expert, eight
// row tiles to a group within one (neighbouring tiles share A rows and B
// columns).  The XCDs, to which the hardware deals workgroups in turn, take one
// stretch each, so that an expert's weights pass through one L2.  `unit`: what
// the caller's segments are multiples of (1 or 32; others are cut down to it).
template <int TILE = BM>
__device__ __forceinline__ bool expert_tile(const int32_t* offsets, int experts, int rows, int unit, int tiles_n, int pid,
                                            ExpertTile& t) {
  const int lane = threadIdx.x & 63;
  // row tiles of the experts of a turn, two a lane (64 apart, so that their
  // offsets come at once), summed up to and with each
  int lo[2], hi[2], mine[2], sum[2];
  const auto count = [&](int at) {
    int from[2], to[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = at + 64 * h + lane;
      from[h] = offsets[std::min(e, experts)];
      to[h] = offsets[std::min(e + 1, experts)];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) asm volatile("" : "+v"(from[h]), "+v"(to[h]));   // all four in flight before the first use
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = at + 64 * h + lane;
      lo[h] = std::min(std::max(from[h] & -unit, 0), rows);
      const int end = std::min(std::max(to[h] & -unit, lo[h]), rows);
      hi[h] = e < experts ? end : (e == experts ? rows : lo[h]);
      mine[h] = (hi[h] - lo[h] + TILE - 1) / TILE;
    }
    sum[0] = wave_prefix_sum(mine[0]);
    sum[1] = wave_prefix_sum(mine[1]) + __builtin_amdgcn_readlane(sum[0], 63);
    return __builtin_amdgcn_readlane(sum[1], 63);
  };
  int total = 0;
  for (int at = 0; at <= experts; at += 128) total += count(at);
  total *= tiles_n;
  const int share = (total + 7) >> 3, l = (pid & 7) * share + (pid >> 3);
  if ((pid >> 3) >= share || l >= total) return false;
  int before = 0;                                        // row tiles of earlier turns
  for (int at = 0; at <= experts; at += 128) {
    if (experts >= 128) count(at);                       // one turn: as it stands
    const uint64_t first_half = __builtin_amdgcn_ballot_w64(l < (before + sum[0]) * tiles_n);
    const uint64_t behind = first_half ? first_half : __builtin_amdgcn_ballot_w64(l < (before + sum[1]) * tiles_n);
    if (behind) {
      const int src = __builtin_ctzll(behind);
      const auto of = [&](const int (&v)[2]) {
        const int a = __builtin_amdgcn_readlane(v[0], src), b = __builtin_amdgcn_readlane(v[1], src);
        return first_half ? a : b;
      };
      const int tiles_m = of(mine), first = before + of(sum) - tiles_m;
      const int in = l - first * tiles_n, width = 8 * tiles_n, group = in / width;
      const int rest = in - group * width, height = std::min(tiles_m - 8 * group, 8);
      // the divisions run on the vector unit: back to scalar registers
      t.expert = __builtin_amdgcn_readfirstlane(at + (first_half ? 0 : 64) + src);
      t.end = of(hi);
      t.m0 = of(lo) + __builtin_amdgcn_readfirstlane((8 * group + rest % height) * TILE);
      t.tn = __builtin_amdgcn_readfirstlane(rest / height);
      return true;
    }
    before += __builtin_amdgcn_readlane(sum[1], 63);
  }
  return false;
}

// Operands of the products over sorted rows.
struct ExpertsArgs {
  const int32_t* offsets;                                // [experts + 1]
  int experts, rows;
  int64_t n, k;                                          // rows of one expert's weights, their length
  const uint8_t *ac, *as, *bc, *bs;
  const uint8_t *a2c, *a2s, *b2c, *b2s;                  // second pair, or null
};

template <int kMode>
__global__ __launch_bounds__(kFastThreads) void gemm_experts_kernel(ExpertsArgs a, Epilogue e) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmemBytes];
  ExpertTile t;
  if (!expert_tile(a.offsets, a.experts, a.rows, 1, (int)((a.n + BN - 1) / BN), (int)grid_tile(), t)) return;
  const int64_t n0 = (int64_t)t.tn * BN, wc = a.n * (a.k >> 1), ws = a.n * (a.k >> 5);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 2, wn = wave & 3, hl = lane >> 5;
  v16f acc[4][2];
  if (t.expert == a.experts || (kMode == kShort && a.k == 0)) {
    zero_tile(acc);
  } else {
    const Operand A{a.ac, a.as, t.end}, B{a.bc + t.expert * wc, a.bs + t.expert * ws, a.n};
    const Operand A2{a.a2c, a.a2s, t.end}, B2{a.b2c + t.expert * wc, a.b2s + t.expert * ws, a.n};
    main_loop_fast<false, kMode>(smem, A, B, t.m0, n0, 0, a.k, acc, wm, wn, &A2, &B2, k_range(0, (int)(a.k >> 5)));
  }
  store_epilogue<true>(smem, acc, e, t.end, a.n, t.m0, n0, wave, lane, wm, wn, hl);
}

// The same in 64 x 64 tiles.
__global__ __launch_bounds__(kSmallThreads, 3) void gemm_experts_small_kernel(ExpertsArgs a, Epilogue e) {
  __shared__ __attribute__((aligned(16))) float smem[kSmallSmem / sizeof(float)];
  ExpertTile t;
  if (!expert_tile<kSmallTile>(a.offsets, a.experts, a.rows, 1, (int)((a.n + kSmallTile - 1) / kSmallTile), (int)grid_tile(), t)) return;
  const int64_t wc = a.n * (a.k >> 1), ws = a.n * (a.k >> 5);
  const Operand A{a.ac, a.as, t.end}, B{a.bc + t.expert * wc, a.bs + t.expert * ws, a.n};
  const Operand A2{a.a2c, a.a2s, t.end}, B2{a.b2c + t.expert * wc, a.b2s + t.expert * ws, a.n};
  small_tile<true>(smem, A, B, A2, B2, t.m0, (int64_t)t.tn * kSmallTile, a.k, k_range(0, t.expert == a.experts ? 0 : (int)(a.k >> 5)), e);
}

// dW_e = A[:, segment] B[:, segment]^T: rows of A and B hold `tokens` values.
// The K range of a segment starts and ends inside a K step: the loop masks the
// blocks of the neighbours' tokens.  `num`: tiles of all experts.
__global__ __launch_bounds__(kFastThreads) void gemm_experts_wgrad_kernel(
    const int32_t* __restrict__ offsets, int num, int64_t tokens, int64_t M, int64_t N, const uint8_t* __restrict__ ac,
    const uint8_t* __restrict__ as, const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs, Epilogue e) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmemBytes];
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + BN - 1) / BN), tiles = tiles_m * tiles_n;
  // The XCDs take the tiles in turns of eight neighbours, 4 x 2 blocks that share
  // operands: every XCD has its share of every expert, whose K ranges differ in
  // length.  (64 experts, 2048 x 2048, 1024 tokens each on average, spread as e^N(0,
  // 1/2): 306 us; in turns of 32 328, in one stretch an XCD 324, 8 x 1 blocks 325.
  // Where all are as long, one stretch of 4 x 8 blocks is faster: 291 against 301.)
  if (grid_tile() >= num) return;
  const int pid = (int)grid_tile(), turn = pid >> 6, l = turn == num >> 6 ? pid : (turn << 6) + ((pid & 7) << 3) + ((pid >> 3) & 7);
  const int expert = l / tiles, in = l - expert * tiles;
  const int group = in / (4 * tiles_n), rest = in - group * 4 * tiles_n, height = std::min(tiles_m - 4 * group, 4);
  const int64_t m0 = (int64_t)(4 * group + rest % height) * BM, n0 = (int64_t)(rest / height) * BN;
  const int blocks = (int)(tokens >> 5);
  const int lo = std::min(std::max(offsets[expert] >> 5, 0), blocks), hi = std::min(std::max(offsets[expert + 1] >> 5, lo), blocks);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 2, wn = wave & 3, hl = lane >> 5;
  v16f acc[4][2];
  if (hi == lo) {
    if (e.accumulate) return;
    zero_tile(acc);
  } else {
    const Operand A{ac, as, M}, B{bc, bs, N};
    main_loop_fast<false, kWindow>(smem, A, B, m0, n0, 0, tokens, acc, wm, wn, nullptr, nullptr, k_range(lo, hi));
  }
  e.y = e.y_f32 ? static_cast<void*>(static_cast<float*>(e.y) + expert * M * N)
                : static_cast<void*>(static_cast<uint16_t*>(e.y) + expert * M * N);
  store_epilogue<true>(smem, acc, e, M, N, m0, n0, wave, lane, wm, wn, hl);
}

// The same in 64 x 64 tiles, an expert's in turn.
__global__ __launch_bounds__(kSmallThreads, 3) void gemm_experts_wgrad_small_kernel(
    const int32_t* __restrict__ offsets, int64_t tokens, int64_t M, int64_t N, const uint8_t* __restrict__ ac,
    const uint8_t* __restrict__ as, const uint8_t* __restrict__ bc, const uint8_t* __restrict__ bs, Epilogue e) {
  __shared__ __attribute__((aligned(16))) float smem[kSmallSmem / sizeof(float)];
  const int tiles_m = (int)((M + kSmallTile - 1) / kSmallTile), tiles = tiles_m * (int)((N + kSmallTile - 1) / kSmallTile);
  const int expert = blockIdx.x / tiles, in = blockIdx.x - expert * tiles, blocks = (int)(tokens >> 5);
  const int lo = std::min(std::max(offsets[expert] >> 5, 0), blocks), hi = std::min(std::max(offsets[expert + 1] >> 5, lo), blocks);
  if (hi == lo && e.accumulate) return;
  const Operand A{ac, as, M}, B{bc, bs, N}, none{};
  e.y = e.y_f32 ? static_cast<void*>(static_cast<float*>(e.y) + expert * M * N)
                : static_cast<void*>(static_cast<uint16_t*>(e.y) + expert * M * N);
  small_tile<true>(smem, A, B, none, none, (int64_t)(in % tiles_m) * kSmallTile, (int64_t)(in / tiles_m) * kSmallTile, tokens,
                   k_range(lo, hi), e);
}

struct SwigluOut {
  uint16_t *a, *b;
  uint8_t *h_codes, *h_scales, *ht_codes, *ht_scales;
  uint32_t signs;
};

// n: FFN columns; an expert's weights are its W1 rows and then its W3 rows.
template <int kMode>
__global__ __launch_bounds__(kFastThreads) void swiglu_experts_kernel(ExpertsArgs a, SwigluOut o) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kSmemBytes];
  ExpertTile t;
  if (!expert_tile(a.offsets, a.experts, a.rows, 32, (int)((a.n + 127) / 128), (int)grid_tile(), t)) return;
  const int64_t n0 = (int64_t)t.tn * 128, wc = a.n * a.k, ws = a.n * (a.k >> 4);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 2, wn = wave & 3, hl = lane >> 5;
  v16f acc[4][2];
  if (t.expert == a.experts || (kMode == kShort && a.k == 0)) {
    zero_tile(acc);
  } else {
    const Operand A{a.ac, a.as, t.end}, B{a.bc + t.expert * wc, a.bs + t.expert * ws, 2 * a.n};
    main_loop_fast<true, kMode>(smem, A, B, t.m0, n0, a.n, a.k, acc, wm, wn, nullptr, nullptr, k_range(0, (int)(a.k >> 5)));
  }
  swiglu_epilogue_staged(smem, acc, t.end, a.rows, a.n, t.m0, n0, wave, lane, wm, wn, hl, o.a, o.b, o.h_codes, o.h_scales,
                         o.ht_codes, o.ht_scales, o.signs);
}

// Workgroups of a product over sorted rows: the row tiles that any segments of
// so many rows can make (a segment's last tile may be all but empty, and so may
// that of the rows behind the last), times the column tiles, in eights (one of
// each for an XCD); -1 past kMostTiles.
static int64_t experts_grid(int64_t rows, int64_t experts, int64_t n, int64_t bn, int64_t bm = BM) {
  if (n > kMaxExpertRows) return -1;
  const int64_t tm = rows / bm + std::min(experts + 1, rows), tn = (n + bn - 1) / bn;
  return tm > kMostTiles / tn ? -1 : (tm * tn + 7) / 8 * 8;
}

// Workgroups in 64 x 64 tiles, or 0 where the large ones are faster.  The small ones
// are where they are few, the padding's and the last rows' counted (large and small:
// 232 of them 7.5 and 4.5 us, 712 9.9 and 6.5, 1088 37 and 34, 1344 37 and 38, 1856 22
// and 26), and where the experts have few rows, which fill a small part of a large tile:
// 80 rows an expert, padding counted (64 experts' 2048 x 2048: 40 rows 48 and 42 us, 96
// rows 60 and 59, 128 rows 64 and 72), or 48 where rows of W of more than 2048 values
// and large tiles for every CU leave little of their start bare (8 experts' 14336 x
// 4096: 8 rows 64 and 58 us, 64 rows 71 and 85, 96 rows 80 and 111; 16 experts' 4096 x
// 4096: 48 rows 61 and 50, 64 rows 45 and 57).  Over 148 calls with operands from memory
// this is 0.8% above the better of the two, at most 16%.
static int64_t experts_small_grid(int64_t rows, int64_t experts, int64_t n, int64_t k) {
  const int64_t grid = experts_grid(rows, experts, n, kSmallTile, kSmallTile);
  const int64_t few = k > 2048 && experts * ((n + BN - 1) / BN) >= 256 ? 48 : 80;
  return grid > 0 && (grid <= 1200 || rows <= few * experts) ? grid : 0;
}

// The most 64 x 64 tiles of the experts' weight gradients together (large and small,
// operands from memory: 4 experts' 128 x 128, 65536 tokens in all, 16 small tiles, 90
// and 39 us; 16 experts' 32 x 1024, 32768, 256 tiles, 31 and 14; 64 experts' 256 x 256,
// 65536, 1024 tiles, 43 and 24; 4 experts' 1024 x 1024, 32768, 1024 tiles, 65 and 62 (50
// and 54 from the caches); 5 experts' 1024 x 1024, 16384, 1280 tiles, 48 and 38; 3
// experts' 1408 x 1408, 16384, 1452 tiles, 54 and 59; 8 experts' 1024 x 1024, 2048, 2048
// tiles, 16.5 and 16.9; 64 experts' 512 x 512, 65536, 4096 tiles, 53 and 60).
constexpr int64_t kSmallGradients = 1024;

static bool operands_aligned(const uint8_t* c, const uint8_t* s) { return aligned16(c) && aligned16(s); }

}  // namespace mx

using namespace mx;

extern "C" {

fp4_status fp4_gemm_experts(int64_t experts, int64_t rows, int64_t n, int64_t k, const int32_t* offsets,
                            const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                            const uint8_t* b_scales, const uint8_t* a2_codes, const uint8_t* a2_scales,
                            const uint8_t* b2_codes, const uint8_t* b2_scales, void* c, fp4_dtype c_type, int64_t ldc,
                            hipStream_t stream) {
  if (!dtype_ok(c_type)) return FP4_EINVAL;
  if (!experts_ok(experts) || rows < 0 || !mult32z(n) || !mult32z(k) || k >= ((int64_t)1 << 24) || ldc < n) return FP4_ESHAPE;
  if (rows == 0 || n == 0) return FP4_OK;
  if (rows > kMaxExpertRows) return FP4_ESHAPE;
  const bool pair = a2_codes || a2_scales || b2_codes || b2_scales;
  if (!offsets || !c || (k > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) ||
      (pair && !(a2_codes && a2_scales && b2_codes && b2_scales)))
    return FP4_EINVAL;
  const int64_t grid = experts_grid(rows, experts, n, BN);
  if (grid < 0) return FP4_ESHAPE;
  if (!operands_aligned(a_codes, a_scales) || !operands_aligned(b_codes, b_scales) || !operands_aligned(a2_codes, a2_scales) ||
      !operands_aligned(b2_codes, b2_scales) || !aligned16(c) || ldc % (c_type == FP4_F32 ? 4 : 8) != 0 ||
      (reinterpret_cast<uintptr_t>(offsets) & 3))
    return FP4_EALIGN;
  const ExpertsArgs a{offsets, (int)experts, (int)rows, n, k, a_codes, a_scales, b_codes, b_scales, a2_codes, a2_scales,
                      b2_codes, b2_scales};
  Epilogue e{};
  e.y = c;
  e.ldy = ldc;
  e.y_f32 = c_type == FP4_F32;
  e.stream = streams(rows, n * (e.y_f32 ? 4 : 2));
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, tile_grid(grid), dim3(kFastThreads), 0, as_stream(stream), a, e);
  };
  const int64_t small = experts_small_grid(rows, experts, n, k);
  if (small > 0) {
    hipLaunchKernelGGL(gemm_experts_small_kernel, tile_grid(small), dim3(kSmallThreads), 0, as_stream(stream), a, e);
    return launch_status();
  }
  const int mode = k_mode(k);
  if (mode == kWhole) go(gemm_experts_kernel<kWhole>);
  else if (mode == kWindow) go(gemm_experts_kernel<kWindow>);
  else go(gemm_experts_kernel<kShort>);
  return launch_status();
}

fp4_status fp4_gemm_experts_wgrad(int64_t experts, int64_t tokens, int64_t m, int64_t n, const int32_t* offsets,
                                  const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                                  const uint8_t* b_scales, void* c, fp4_dtype c_type, int accumulate, hipStream_t stream) {
  if (!dtype_ok(c_type) || (accumulate != 0 && accumulate != 1) || (accumulate && c_type != FP4_F32)) return FP4_EINVAL;
  if (!experts_ok(experts) || tokens < 0 || tokens % 256 != 0 || tokens >= ((int64_t)1 << 24) || !mult32z(m) || !mult32z(n))
    return FP4_ESHAPE;
  if (m == 0 || n == 0) return FP4_OK;
  if (!offsets || !c || (tokens > 0 && (!a_codes || !a_scales || !b_codes || !b_scales))) return FP4_EINVAL;
  const int64_t tiles = tiles_of(m, BM, n, BN);
  if (tiles < 0 || tiles > kMostTiles / experts) return FP4_ESHAPE;
  if (!operands_aligned(a_codes, a_scales) || !operands_aligned(b_codes, b_scales) || !aligned16(c) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3))
    return FP4_EALIGN;
  Epilogue e{};
  e.y = c;
  e.ldy = n;
  e.y_f32 = c_type == FP4_F32;
  e.accumulate = accumulate;
  e.stream = streams(experts * m, n * (e.y_f32 ? 4 : 2));
  const int64_t small = tiles_of(m, kSmallTile, n, kSmallTile) * experts;
  if (small > 0 && small <= kSmallGradients) {   // below 0: more tiles than a launch holds
    hipLaunchKernelGGL(gemm_experts_wgrad_small_kernel, dim3((unsigned)small), dim3(kSmallThreads), 0, as_stream(stream),
                       offsets, tokens, m, n, a_codes, a_scales, b_codes, b_scales, e);
    return launch_status();
  }
  hipLaunchKernelGGL(gemm_experts_wgrad_kernel, tile_grid(tiles * experts), dim3(kFastThreads), 0, as_stream(stream),
                     offsets, (int)(tiles * experts), tokens, m, n, a_codes, a_scales, b_codes, b_scales, e);
  return launch_status();
}

fp4_status fp4_swiglu_producer_experts(int64_t experts, int64_t rows, int64_t f, int64_t d, const int32_t* offsets,
                                       const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w13_codes,
                                       const uint8_t* w13_scales, uint16_t* a_bf16, uint16_t* b_bf16, uint8_t* h_codes,
                                       uint8_t* h_scales, uint8_t* ht_codes, uint8_t* ht_scales, uint32_t sign_mask16,
                                       hipStream_t stream) {
  if ((ht_codes == nullptr) != (ht_scales == nullptr)) return FP4_EINVAL;
  if (!experts_ok(experts) || !mult32z(rows) || !mult32z(f) || !mult32z(d) || d >= ((int64_t)1 << 24)) return FP4_ESHAPE;
  if (rows == 0 || f == 0) return FP4_OK;
  if (rows > kMaxExpertRows) return FP4_ESHAPE;
  if (!offsets || !a_bf16 || !b_bf16 || !h_codes || !h_scales ||
      (d > 0 && (!x_codes || !x_scales || !w13_codes || !w13_scales)))
    return FP4_EINVAL;
  const int64_t grid = experts_grid(rows, experts, f, 128);
  if (grid < 0) return FP4_ESHAPE;
  if (!operands_aligned(x_codes, x_scales) || !operands_aligned(w13_codes, w13_scales) || !aligned16(h_codes) ||
      !aligned16(a_bf16) || !aligned16(b_bf16) || !aligned16(ht_codes) || (reinterpret_cast<uintptr_t>(offsets) & 3))
    return FP4_EALIGN;
  const ExpertsArgs a{offsets, (int)experts, (int)rows, f, d, x_codes, x_scales, w13_codes, w13_scales, nullptr, nullptr,
                      nullptr, nullptr};
  const SwigluOut o{a_bf16, b_bf16, h_codes, h_scales, ht_codes, ht_scales, sign_mask16 & 0xFFFFu};
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, tile_grid(grid), dim3(kFastThreads), 0, as_stream(stream), a, o);
  };
  const int mode = k_mode(d);
  if (mode == kWhole) go(swiglu_experts_kernel<kWhole>);
  else if (mode == kWindow) go(swiglu_experts_kernel<kWindow>);
  else go(swiglu_experts_kernel<kShort>);
  return launch_status();
}

}  // extern "C"
