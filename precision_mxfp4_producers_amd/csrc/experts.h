// Limits shared by the calls on tokens sorted by expert.
#pragma once

#include <stdint.h>

namespace mx {

constexpr int64_t kMaxExperts = 1024;                    // one a thread of the sort's workgroup
constexpr int64_t kMaxExpertRows = (int64_t)1 << 30;     // 32-bit row indices

inline bool experts_ok(int64_t e) { return e >= 1 && e <= kMaxExperts; }

}  // namespace mx
