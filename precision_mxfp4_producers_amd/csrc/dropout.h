// Counter-based dropout shared by fp4_dropout and the RMSNorm producer and its
// backward: the mask is a function of (seed, offset) and the element's index
// and is never stored.
//
// Element c of row r has index i = r * 8 ceil(cols / 8) + c, so that a group
// of eight consecutive columns is one Philox4x32-10 block (128 bits): block
// i >> 3, element i & 7 taking half (i & 1) of word (i >> 1) & 3.  It is kept
// iff its 16-bit half is >= thr = floor(65536 p + 1/2), and kept values are
// multiplied by RN(65536 / (65536 - thr)), the inverse of the probability that
// the 16 bits give.  Sixteen bits an element, and not the 32 that the
// stochastic rounding takes, halve the generator's integer multiplies, which
// bound the producers that draw; p is then a multiple of 2^-16.
#pragma once

#include "mx_device.h"

namespace mx {

struct Dropout {
  uint32_t thr;                                          // 0: off, 65536: everything dropped
  float scale;                                           // of the kept values (0 when nothing is kept)
  uint64_t seed, offset;
};

// Host side: p in [0, 1] (checked by the caller).
inline Dropout make_dropout(float p, uint64_t seed, uint64_t offset) {
  const uint32_t thr = (uint32_t)((double)p * 65536.0 + 0.5);
  return {thr, thr < 65536u ? (float)(65536.0 / (double)(65536u - thr)) : 0.0f, seed, offset};
}

// Applies the mask to eight consecutive elements (Philox block blk) and adds
// `base` (null: nothing): v = keep ? v * scale + base : base.  A dropped
// element is selected away, not multiplied by zero, so an infinity or NaN
// under the mask leaves no trace; the kept one takes one fused multiply-add,
// one rounding.
__device__ __forceinline__ void dropout8(float (&v)[8], const float* base, uint64_t blk, const Dropout& d) {
  const u32x4 w = sr_words(blk, d.seed, d.offset);
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = (j & 1) ? (q[j >> 1] >> 16) : (q[j >> 1] & 0xFFFFu);
    const float kept = base ? __builtin_fmaf(v[j], d.scale, base[j]) : __fmul_rn(v[j], d.scale);
    v[j] = h >= d.thr ? kept : (base ? base[j] : 0.0f);
  }
}

}  // namespace mx
