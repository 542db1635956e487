// Limits and the lookup of segments shared by the calls on tokens sorted by
// expert.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

constexpr int64_t kMaxExperts = 1024;                    // one a thread of the sort's workgroup
constexpr int64_t kMaxExpertRows = (int64_t)1 << 30;     // 32-bit row indices

// Sum of the lanes' values up to and with each lane's (all lanes active): steps
// of 1, 2, 4 and 8 within rows of 16 lanes, then rows into the rows behind them.
template <typename T>
__device__ __forceinline__ T wave_prefix_sum(T x) {
  static_assert(sizeof(T) == 4, "one register");
  int v = (int)x;
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast 15: rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast 31: rows 2 and 3
  return (T)v;
}

inline bool experts_ok(int64_t e) { return e >= 1 && e <= kMaxExperts; }

}  // namespace mx
