// Tokens sorted by expert and back: the sorted order (fp4_expert_sort), the
// activations in it with their codes (fp4_expert_gather), the experts' results
// weighted and added per token (fp4_expert_combine) and that sum's gradients
// (fp4_expert_combine_backward).
//
// A slot is one of a token's k choices, slot t k + j.  Expert e owns the sorted
// rows offsets[e] .. offsets[e + 1] - 1: its slots in ascending order, then
// padding to a multiple of `align` (32: the column-facing codes hold blocks of
// 32 tokens, none of which may mix two experts).
//
// Method: "Format-Aware Fusion for Fast FP4 Pretraining", §2.3 (Eq. 6: token
// blocks of the column-facing codes), §3.1 (a boundary leaves the operands that
// its consumer reads).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "abi_common.h"
#include "experts.h"
#include "rows.h"

namespace mx {

// ---------------------------------------------------------------- sort
struct SortArgs {
  const void* ids;                                       // [slots] int32 or int64
  int slots, experts, align, capacity;
  int chunk;                                             // slots of a workgroup
  int32_t *offsets, *out_slots, *rows;
  uint32_t* counts;                                      // [workgroups][experts] (several workgroups)
};

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

// The expert of slot s, or -1.
template <bool I64>
__device__ __forceinline__ int slot_expert(const SortArgs& a, int s) {
  if constexpr (I64) {
    const int64_t v = static_cast<const int64_t*>(a.ids)[s];
    return v >= 0 && v < a.experts ? (int)v : -1;
  } else {
    const int32_t v = static_cast<const int32_t*>(a.ids)[s];
    return (uint32_t)v < (uint32_t)a.experts ? v : -1;
  }
}

// This workgroup's slots counted by wave and expert: counts[w * experts + e].
template <bool I64>
__device__ __forceinline__ void count_slots(const SortArgs& a, uint32_t* counts, int first, int last, int part) {
  for (int i = threadIdx.x; i < kSortWaves * a.experts; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int begin = first + wave * part, end = std::min(begin + part, last);
  for (int s = begin + lane; s < end; s += 64) {
    const int e = slot_expert<I64>(a, s);
    if (e >= 0) atomicAdd(&counts[wave * a.experts + e], 1u);
  }
  __syncthreads();
}

template <bool I64>
__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortArgs a) {
  __shared__ uint32_t counts[kSortWaves * kMaxExperts];
  const int first = blockIdx.x * a.chunk, last = std::min(first + a.chunk, a.slots);
  count_slots<I64>(a, counts, first, last, a.chunk / kSortWaves);
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    uint32_t n = 0;
    for (int w = 0; w < kSortWaves; ++w) n += counts[w * a.experts + e];
    a.counts[(int64_t)blockIdx.x * a.experts + e] = n;
  }
}

// Order within an expert is that of the slots, with no atomics: a workgroup
// takes a stretch of slots, a wave a stretch of those, 64 slots at a time, and
// a slot's row is the expert's first row, plus the expert's slots in earlier
// workgroups, waves and turns, plus those in lower lanes (found by comparing
// the expert's bits across the wave).  Latency: 65536 slots of 64 experts take
// 4.7 (count) and 6.6 us (32 workgroups), two slots 2.8 (one, no count).
template <bool I64>
__global__ __launch_bounds__(kSortThreads) void expert_sort_kernel(SortArgs a) {
  __shared__ uint32_t counts[kSortWaves * kMaxExperts];   // [waves][experts]
  __shared__ uint32_t wave_sum[kSortWaves];
  __shared__ uint32_t total_rows;
  const int first = blockIdx.x * a.chunk, last = std::min(first + a.chunk, a.slots);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, part = a.chunk / kSortWaves;
  count_slots<I64>(a, counts, first, last, part);
  // thread e: its expert's slots in all workgroups, and in the earlier ones
  const int e = threadIdx.x;
  uint32_t before = 0, total = 0;
  if (e < a.experts) {
    if (gridDim.x > 1) {
#pragma unroll 8
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const uint32_t n = a.counts[(int64_t)b * a.experts + e];
        if (b < (int)blockIdx.x) before += n;
        total += n;
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += counts[w * a.experts + e];
    }
  }
  // first row of the expert: sum of the padded totals of the earlier ones
  const uint32_t padded = (total + a.align - 1) / a.align * a.align;
  const uint32_t sum = wave_prefix_sum(padded);
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  uint32_t start = sum - padded;
  for (int w = 0; w < wave; ++w) start += wave_sum[w];
  if (e == kSortThreads - 1) total_rows = start + padded;
  if (e < a.experts) {
    uint32_t at = start + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t n = counts[w * a.experts + e];
      counts[w * a.experts + e] = at;
      at += n;
    }
    if (blockIdx.x == 0) a.offsets[e] = (int32_t)start;
    // padding of this expert: the workgroups take the experts in turn
    if (e % (int)gridDim.x == (int)blockIdx.x)
      for (uint32_t r = start + total; r < start + padded; ++r) a.out_slots[r] = -1;
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = (int32_t)total_rows;
  for (int64_t r = total_rows + blockIdx.x * kSortThreads + threadIdx.x; r < a.capacity; r += gridDim.x * kSortThreads)
    a.out_slots[r] = -1;
  const int begin = first + wave * part, end = std::min(begin + part, last);
  const int bits = 32 - __builtin_clz(std::max(a.experts - 1, 1));
  uint32_t* const mine = counts + wave * a.experts;
  for (int s0 = begin; s0 < end; s0 += 64) {
    const int s = s0 + lane;
    const int x = s < end ? slot_expert<I64>(a, s) : -1;
    uint64_t same = __builtin_amdgcn_ballot_w64(x >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __builtin_amdgcn_ballot_w64((x >> b) & 1);
      same &= (x >> b) & 1 ? set : ~set;
    }
    const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    uint32_t row = 0xFFFFFFFFu;
    if (x >= 0) row = mine[x] + rank;
    // all lanes have read before one of them moves the count on
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if (x >= 0 && rank == 0) mine[x] = row + __builtin_popcountll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if (s < end) a.rows[s] = (int32_t)row;
    if (x >= 0) a.out_slots[row] = s;
  }
}

// ---------------------------------------------------------------- gather
struct GatherArgs {
  const uint16_t* x;                                     // [t][ldx]
  int64_t ldx;
  const int32_t* slots;                                  // [rows]
  int rows, t, k, d;
  uint16_t* xs;                                          // [rows][d], or null
  uint8_t *codes, *scales;                               // or null
  int e4m3;
  int stream;                                            // xs past the caches
  int32_t* where;                                        // [t][k] rows of the slots (by tokens)
  int token_groups;                                      // workgroups that take tokens
};

// The token of a row's slot, or -1.
__device__ __forceinline__ int row_token(const GatherArgs& a, int slot) {
  const int token = slot >= 0 ? slot / a.k : -1;
  return token < a.t ? token : -1;
}

// Codes and scale of eight values, four neighbouring lanes a block of 32.
struct Coded {
  uint2 codes;                                           // E2M1: the first word
  int e;
};
__device__ __forceinline__ Coded encode8(const GatherArgs& a, const uint4 v) {
  const uint32_t am = max_quad(bf16_absmax8(v.x, v.y, v.z, v.w)) << 16;
  const int e = a.e4m3 ? upward_exp_e4m3(am) : upward_exp(am);
  return Coded{a.e4m3 ? e4m3_8(v, pow2_scale(e)) : make_uint2(rtn8_bf16(v.x, v.y, v.z, v.w, pow2_scale(e)), 0u), e};
}

// Columns c .. c + 7 of row r.
__device__ __forceinline__ void put_gathered(const GatherArgs& a, int64_t r, int c, const uint4 v, const Coded& q) {
  if (a.xs) put(reinterpret_cast<u32x4v*>(a.xs + r * a.d + c), u32x4v{v.x, v.y, v.z, v.w}, a.stream);
  if (a.codes) {
    if (a.e4m3) *reinterpret_cast<uint2*>(a.codes + r * a.d + c) = q.codes;
    else *reinterpret_cast<uint32_t*>(a.codes + r * (a.d >> 1) + (c >> 1)) = q.codes.x;
    if ((threadIdx.x & 3) == 0) a.scales[r * (a.d >> 5) + (c >> 5)] = (uint8_t)(q.e + 127);
  }
}

// Row r whole, by G lanes, of which this is lane i: a token's activations, or
// zeros.
template <int G>
__device__ __forceinline__ void gather_row(const GatherArgs& a, int64_t r, int token, int i) {
  const uint16_t* const x = a.x + (int64_t)std::max(token, 0) * a.ldx;
  for (int c0 = i * 8; c0 < a.d; c0 += 4 * G * 8) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = make_uint4(0, 0, 0, 0);
    if (token >= 0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const uint4*>(x + std::min(c0 + u * G * 8, a.d - 8));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u * G * 8;
      if (c >= a.d) break;                               // whole groups of four lanes
      put_gathered(a, r, c, v[u], a.codes ? encode8(a, v[u]) : Coded{});
    }
  }
}

// Row by row, 2^LG lanes a row: one launch.
template <int LG>
__global__ __launch_bounds__(256) void expert_gather_kernel(GatherArgs a) {
  constexpr int G = 1 << LG;
  for (int64_t r = (int64_t)blockIdx.x * (256 / G) + (threadIdx.x >> LG); r < a.rows; r += (int64_t)gridDim.x * (256 / G))
    gather_row<G>(a, r, row_token(a, a.slots[r]), threadIdx.x & (G - 1));
}

// By tokens: x is read and encoded once for all of a token's rows, where rows in
// their order would bring it from the Infinity Cache once for each (8192 tokens x
// 2048 to eight rows each, 277 MB of rows: 76 us by rows, 61 by tokens).  The rows
// of the slots come first:
__global__ __launch_bounds__(256) void expert_where_kernel(GatherArgs a) {
  for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < a.rows; r += (int64_t)gridDim.x * 256) {
    const int s = a.slots[r];
    if (row_token(a, s) >= 0) a.where[s] = (int32_t)r;
  }
}

// (4.7 us) and then a wave takes 2048 columns of a token to all its rows: those
// without codes, 311 MB in 59 us, 5.3 TB/s, as a copy does.  where[s] may hold
// anything if no row has slot s, and holds one of them if several have: a row
// counts as the slot's if its slot is that.  The workgroups behind those of the
// tokens take the rows that are no slot's: those without a token, and others than
// where[s] with slot s.
__global__ __launch_bounds__(256) void expert_scatter_kernel(GatherArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if ((int)blockIdx.x >= a.token_groups) {
    // a wave's rows lie apart, so that a run of padding is many waves'
    const int64_t waves = ((int64_t)gridDim.x - a.token_groups) * 4, first = ((int64_t)blockIdx.x - a.token_groups) * 4 + wave;
    for (int64_t r0 = first; r0 < a.rows; r0 += waves * 64) {
      const int64_t r = r0 + lane * waves;
      int token = -1;
      bool mine = false;
      if (r < a.rows) {
        const int s = a.slots[r];
        token = row_token(a, s);
        mine = token < 0 || a.where[s] != r;
      }
      for (uint64_t left = __builtin_amdgcn_ballot_w64(mine); left; left &= left - 1) {
        const int l = __builtin_ctzll(left);
        gather_row<64>(a, r0 + l * waves, __builtin_amdgcn_readlane(token, l), lane);
      }
    }
    return;
  }
  const int parts = (a.d + 2047) / 2048;
  for (int64_t q = (int64_t)blockIdx.x * 4 + wave; q < (int64_t)a.t * parts; q += (int64_t)a.token_groups * 4) {
    const int token = (int)(q / parts), first = (int)(q - (int64_t)token * parts) * 2048 + lane * 8;
    uint4 v[4];
    Coded e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const uint4*>(a.x + token * a.ldx + std::min(first + u * 512, a.d - 8));
#pragma unroll
    for (int u = 0; u < 4; ++u) e[u] = a.codes ? encode8(a, v[u]) : Coded{};
    for (int j0 = 0; j0 < a.k; j0 += 64) {
      int row = -1;
      if (j0 + lane < a.k) {
        const int s = token * a.k + j0 + lane;
        row = a.where[s];
        if ((uint32_t)row >= (uint32_t)a.rows || a.slots[row] != s) row = -1;
      }
      for (uint64_t left = __builtin_amdgcn_ballot_w64(row >= 0); left; left &= left - 1) {
        const int64_t r = __builtin_amdgcn_readlane(row, __builtin_ctzll(left));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (first + u * 512 < a.d) put_gathered(a, r, first + u * 512, v[u], e[u]);
      }
    }
  }
}

// ---------------------------------------------------------------- combine
struct CombineArgs {
  const void* z;                                         // [rows][ldz] bf16 or fp32
  int64_t ldz;
  const int32_t* where;                                  // [t][k] sorted rows
  const float* weights;                                  // [t][k], or null: all 1
  const uint16_t* residual;                              // [t][ldr], or null
  int64_t ldr;
  uint16_t* out;                                         // [t][ldo]
  int64_t ldo;
  int t, k, d, rows;
};

template <bool F32>
__device__ __forceinline__ void load8_cached(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float4* const f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), v);
  }
}

// One thread per eight columns of a token, four of its rows in flight.  Bound by
// memory: 8192 tokens x 4096 of two bf16 rows each, 268 MB, take 50 us, 5.4 TB/s.
template <bool F32>
__global__ __launch_bounds__(256) void expert_combine_kernel(CombineArgs a) {
  const int per = a.d >> 3;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < (int64_t)a.t * per; q += (int64_t)gridDim.x * 256) {
    const int64_t t = q / per;
    const int c = (int)(q - t * per) * 8;
    float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      float v[4][8], w[4];
      bool live[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = std::min(j0 + u, a.k - 1);
        const int row = a.where[t * a.k + j];
        live[u] = j0 + u < a.k && (uint32_t)row < (uint32_t)a.rows;
        w[u] = a.weights ? a.weights[t * a.k + j] : 1.0f;
        load8_cached<F32>(a.z, (live[u] ? row : 0) * a.ldz + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = live[u] ? __builtin_fmaf(w[u], v[u][i], acc[i]) : acc[i];
    }
    if (a.residual) {
      float b[8];
      unpack8(load_once_u4(a.residual + t * a.ldr + c), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], b[i]);
    }
    *reinterpret_cast<uint4*>(a.out + t * a.ldo + c) = pack8(acc);
  }
}

struct CombineGradArgs {
  const void* dy;                                        // [t][lddy]
  int64_t lddy;
  const void* z;                                         // [rows][ldz]
  int64_t ldz;
  const int32_t* slots;                                  // [rows]
  const int32_t* where;                                  // [t][k]
  const float* weights;                                  // [t][k]
  uint16_t* dz;                                          // [rows][d]
  float* dw;                                             // [t][k]
  int t, k, d, rows;
  int slot_groups;                                       // workgroups that take slots
};

// dz[r] = w dy[t] and dw = <dy[t], z[r]>: a wave a slot, so that a token's waves
// read dy from the cache; the workgroups behind them clear the rows without a
// token.  Bound by memory: 8192 tokens x 2048, eight rows each, 579 MB, take 113
// us, 5.1 TB/s (dz past the caches was slower).
template <bool DYF32, bool ZF32>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(CombineGradArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if ((int)blockIdx.x >= a.slot_groups) {
    // a wave's rows lie apart, so that a run of padding is many waves'
    const int64_t waves = ((int64_t)gridDim.x - a.slot_groups) * 4;
    for (int64_t r0 = ((int64_t)blockIdx.x - a.slot_groups) * 4 + wave; r0 < a.rows; r0 += waves * 64) {
      const int64_t mine = r0 + lane * waves;
      const bool clear = mine < a.rows && (uint32_t)a.slots[mine] >= (uint32_t)(a.t * a.k);
      for (uint64_t left = __builtin_amdgcn_ballot_w64(clear); left; left &= left - 1) {
        const int64_t r = r0 + __builtin_ctzll(left) * waves;
        for (int c = lane * 8; c < a.d; c += 512) *reinterpret_cast<uint4*>(a.dz + r * a.d + c) = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  for (int64_t s = (int64_t)blockIdx.x * 4 + wave; s < (int64_t)a.t * a.k; s += (int64_t)a.slot_groups * 4) {
    const int row = a.where[s];
    if ((uint32_t)row >= (uint32_t)a.rows) {
      if (lane == 0) a.dw[s] = 0.0f;
      continue;
    }
    const int64_t t = s / a.k;
    const float w = a.weights[s];
    float dot = 0.0f;
    for (int c = lane * 8; c < a.d; c += 512) {
      float y[8], z[8], o[8];
      load8_cached<DYF32>(a.dy, t * a.lddy + c, y);
      load8_cached<ZF32>(a.z, row * a.ldz + c, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = __builtin_fmaf(y[i], z[i], dot);
        o[i] = __fmul_rn(w, y[i]);
      }
      *reinterpret_cast<uint4*>(a.dz + (int64_t)row * a.d + c) = pack8(o);
    }
#pragma unroll
    for (int st = 1; st < 64; st <<= 1) dot = __fadd_rn(dot, __shfl_xor(dot, st, 64));
    if (lane == 0) a.dw[s] = dot;
  }
}

// ---------------------------------------------------------------- host side
// Workgroups of a launch (a dimension holds less than 2^32 threads); beyond,
// they walk the work.
constexpr int64_t kMostGroups = 1 << 22;

// Workgroups of the sort and slots of each: one for a few thousand slots, which
// then takes one launch.
static int sort_groups(int64_t slots, int64_t& chunk) {
  constexpr int64_t kOne = 8192, kMost = 256;
  int64_t groups = slots <= kOne ? 1 : std::min((slots + 2047) / 2048, kMost);
  chunk = std::max<int64_t>((slots + groups - 1) / groups + kSortThreads - 1, kSortThreads) / kSortThreads * kSortThreads;
  return (int)std::max<int64_t>((slots + chunk - 1) / chunk, 1);
}

static bool gather_shape_ok(int64_t t, int64_t k, int64_t d, int64_t rows) {
  return t >= 0 && k >= 1 && k <= kMaxExpertRows && t <= kMaxExpertRows / k && mult32z(d) && d <= kMaxExpertRows && rows >= 0 &&
         rows <= kMaxExpertRows + kMaxExperts * 256;
}

// By tokens where the rows outgrow the L2s and a token has several (bf16 rows
// alone, by rows and by tokens: 8 experts a token, 48 MB of rows 11 and 16 us, 66
// MB 21 and 18, 264 MB 76 and 61; 2 a token, 130 MB 41 and 36, with codes 48 and
// 49).
static bool gather_by_tokens(int64_t t, int64_t k, int64_t d, int64_t rows) {
  return t > 0 && k > 1 && d > 128 && rows * d * 2 > ((int64_t)56 << 20);
}

static bool sort_shape_ok(int64_t t, int64_t k, int64_t experts) {
  return t >= 0 && k >= 1 && experts_ok(experts) && k <= kMaxExpertRows && t <= kMaxExpertRows / k;
}

}  // namespace mx

using namespace mx;

extern "C" {

int64_t fp4_expert_capacity(int64_t t, int64_t k, int64_t experts, int64_t align) {
  if (!sort_shape_ok(t, k, experts) || (align != 1 && (align < 32 || align > 256 || align % 32 != 0))) return -1;
  const int64_t slots = t * k;
  if (align == 1) return slots;
  return (slots + std::min(experts, slots) * (align - 1) + 255) / 256 * 256;
}

int64_t fp4_expert_sort_workspace(int64_t t, int64_t k, int64_t experts) {
  if (!sort_shape_ok(t, k, experts)) return -1;
  int64_t chunk;
  const int groups = sort_groups(t * k, chunk);
  return groups > 1 ? groups * experts * (int64_t)sizeof(uint32_t) : 0;
}

fp4_status fp4_expert_sort(int64_t t, int64_t k, int64_t experts, const void* ids, int id_bytes, int64_t align,
                           int64_t capacity, int32_t* offsets, int32_t* slots, int32_t* rows, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
  if (id_bytes != 4 && id_bytes != 8) return FP4_EINVAL;
  const int64_t need = fp4_expert_capacity(t, k, experts, align);
  if (need < 0 || capacity < need || capacity > kMaxExpertRows + kMaxExperts * 256) return FP4_ESHAPE;
  const int64_t ws = fp4_expert_sort_workspace(t, k, experts);
  if (workspace_bytes < ws) return FP4_ESHAPE;
  if (!offsets || (capacity > 0 && !slots) || (t > 0 && (!ids || !rows)) || (ws > 0 && !workspace)) return FP4_EINVAL;
  if ((reinterpret_cast<uintptr_t>(ids) & (id_bytes - 1)) || (reinterpret_cast<uintptr_t>(offsets) & 3) ||
      (reinterpret_cast<uintptr_t>(slots) & 3) || (reinterpret_cast<uintptr_t>(rows) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 3))
    return FP4_EALIGN;
  int64_t chunk;
  const int groups = sort_groups(t * k, chunk);
  const SortArgs a{ids, (int)(t * k), (int)experts, (int)align, (int)capacity, (int)chunk, offsets, slots, rows,
                   static_cast<uint32_t*>(workspace)};
  const auto go = [&](auto count, auto sort) {
    if (groups > 1) {
      hipLaunchKernelGGL(count, dim3(groups), dim3(kSortThreads), 0, as_stream(stream), a);
      const fp4_status st = launch_status();
      if (st != FP4_OK) return st;
    }
    hipLaunchKernelGGL(sort, dim3(groups), dim3(kSortThreads), 0, as_stream(stream), a);
    return launch_status();
  };
  return id_bytes == 8 ? go(expert_count_kernel<true>, expert_sort_kernel<true>)
                       : go(expert_count_kernel<false>, expert_sort_kernel<false>);
}

int64_t fp4_expert_gather_workspace(int64_t t, int64_t k, int64_t d, int64_t rows) {
  if (!gather_shape_ok(t, k, d, rows)) return -1;
  return gather_by_tokens(t, k, d, rows) ? t * k * (int64_t)sizeof(int32_t) : 0;
}

fp4_status fp4_expert_gather(int64_t t, int64_t k, int64_t d, int64_t rows, const uint16_t* x, int64_t ldx,
                             const int32_t* slots, uint16_t* xs, fp4_format format, uint8_t* codes, uint8_t* scales,
                             void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if ((format != FP4_E2M1 && format != FP4_E4M3) || (codes == nullptr) != (scales == nullptr)) return FP4_EINVAL;
  if (!gather_shape_ok(t, k, d, rows) || ldx < d) return FP4_ESHAPE;
  if (rows == 0 || d == 0 || (!xs && !codes)) return FP4_OK;
  if (!slots || (t > 0 && !x)) return FP4_EINVAL;
  const bool by_tokens = gather_by_tokens(t, k, d, rows);
  if (workspace_bytes < fp4_expert_gather_workspace(t, k, d, rows)) return FP4_ESHAPE;
  if (by_tokens && !workspace) return FP4_EINVAL;
  if (!aligned16(x) || !aligned16(xs) || !aligned16(codes) || ldx % 8 != 0 || (reinterpret_cast<uintptr_t>(slots) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 3))
    return FP4_EALIGN;
  GatherArgs a{x, ldx, slots, (int)rows, (int)t, (int)k, (int)d, xs, codes, scales, format == FP4_E4M3,
               streams(rows, d * 2), static_cast<int32_t*>(workspace), 0};
  hipStream_t s = as_stream(stream);
  if (by_tokens) {
    hipLaunchKernelGGL(expert_where_kernel, dim3((unsigned)std::min((rows + 255) / 256, kMostGroups)), dim3(256), 0, s, a);
    const fp4_status st = launch_status();
    if (st != FP4_OK) return st;
    const int64_t tokens = std::min((t * ((d + 2047) / 2048) + 3) / 4, kMostGroups), others = std::min<int64_t>((rows + 31) / 32, 1024);
    a.token_groups = (int)tokens;
    hipLaunchKernelGGL(expert_scatter_kernel, dim3((unsigned)(tokens + others)), dim3(256), 0, s, a);
    return launch_status();
  }
  const auto go = [&](auto kernel, int lg) {
    const int64_t per = 256 >> lg;
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min((rows + per - 1) / per, kMostGroups)), dim3(256), 0, s, a);
  };
  if (d <= 128) go(expert_gather_kernel<4>, 4);
  else go(expert_gather_kernel<6>, 6);
  return launch_status();
}

fp4_status fp4_expert_combine(int64_t t, int64_t k, int64_t d, int64_t rows, const void* z, fp4_dtype z_type, int64_t ldz,
                              const int32_t* where, const float* weights, const uint16_t* residual, int64_t ldr,
                              uint16_t* out, int64_t ldo, hipStream_t stream) {
  if (!dtype_ok(z_type)) return FP4_EINVAL;
  if (t < 0 || t > kMaxExpertRows || k < 1 || k > kMaxExpertRows || t > kMaxExpertRows / k || !mult32z(d) || rows < 0 ||
      rows > kMaxExpertRows + kMaxExperts * 256 || ldz < d || ldo < d || (residual && ldr < d))
    return FP4_ESHAPE;
  if (t == 0 || d == 0) return FP4_OK;
  if (d > kMaxExpertRows) return FP4_ESHAPE;
  const int64_t groups = std::min((t * (d / 8) + 255) / 256, kMostGroups);
  if (!where || !out || (rows > 0 && !z)) return FP4_EINVAL;
  if (!aligned16(z) || !aligned16(residual) || !aligned16(out) || ldz % (z_type == FP4_F32 ? 4 : 8) != 0 || ldo % 8 != 0 ||
      (residual && ldr % 8 != 0) || (reinterpret_cast<uintptr_t>(where) & 3) || (reinterpret_cast<uintptr_t>(weights) & 3))
    return FP4_EALIGN;
  CombineArgs a{z, ldz, where, weights, residual, ldr, out, ldo, (int)t, (int)k, (int)d, (int)rows};
  if (rows == 0) a.k = 0;                                // nothing is routed
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(256), 0, as_stream(stream), a);
  };
  z_type == FP4_F32 ? go(expert_combine_kernel<true>) : go(expert_combine_kernel<false>);
  return launch_status();
}

fp4_status fp4_expert_combine_backward(int64_t t, int64_t k, int64_t d, int64_t rows, const void* dy, fp4_dtype dy_type,
                                       int64_t lddy, const void* z, fp4_dtype z_type, int64_t ldz, const int32_t* slots,
                                       const int32_t* where, const float* weights, uint16_t* dz, float* dw,
                                       hipStream_t stream) {
  if (!dtype_ok(dy_type) || !dtype_ok(z_type)) return FP4_EINVAL;
  if (t < 0 || t > kMaxExpertRows || k < 1 || k > kMaxExpertRows || t > kMaxExpertRows / k || !mult32z(d) ||
      d > kMaxExpertRows || rows < 0 || rows > kMaxExpertRows + kMaxExperts * 256 || lddy < d || ldz < d)
    return FP4_ESHAPE;
  if (t == 0 && rows == 0) return FP4_OK;
  if ((rows > 0 && (!slots || (d > 0 && (!z || !dz)))) || (t > 0 && (!where || !weights || !dw || (d > 0 && !dy))))
    return FP4_EINVAL;
  if (!aligned16(dy) || !aligned16(z) || !aligned16(dz) || lddy % (dy_type == FP4_F32 ? 4 : 8) != 0 ||
      ldz % (z_type == FP4_F32 ? 4 : 8) != 0 || (reinterpret_cast<uintptr_t>(slots) & 3) ||
      (reinterpret_cast<uintptr_t>(where) & 3) || (reinterpret_cast<uintptr_t>(weights) & 3) ||
      (reinterpret_cast<uintptr_t>(dw) & 3))
    return FP4_EALIGN;
  const int64_t groups = std::min((t * k + 3) / 4, kMostGroups), clear = std::min<int64_t>((rows + 31) / 32, 1024);
  const CombineGradArgs a{dy, lddy, z, ldz, slots, where, weights, dz, dw, (int)t, (int)k, (int)d, (int)rows, (int)groups};
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(groups + clear)), dim3(256), 0, as_stream(stream), a);
  };
  if (dy_type == FP4_F32)
    z_type == FP4_F32 ? go(expert_combine_grad_kernel<true, true>) : go(expert_combine_grad_kernel<true, false>);
  else
    z_type == FP4_F32 ? go(expert_combine_grad_kernel<false, true>) : go(expert_combine_grad_kernel<false, false>);
  return launch_status();
}

}  // extern "C"
