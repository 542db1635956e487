// Neighbouring values of a row: loads, stores and E4M3 codes, shared by the
// kernels that hold rows of activations in registers.
#pragma once

#include "mx_device.h"

namespace mx {

// ---------------------------------------------------------------- loads and stores of eight values
__device__ __forceinline__ void unpack8(const uint4 w, float (&v)[8]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? __uint_as_float(q[j >> 1] & 0xFFFF0000u) : __uint_as_float(q[j >> 1] << 16);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16_pack2_rne(v[0], v[1]), bf16_pack2_rne(v[2], v[3]), bf16_pack2_rne(v[4], v[5]),
                    bf16_pack2_rne(v[6], v[7]));
}

template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float* f = static_cast<const float*>(p) + i;
    const uint4 a = load_once_u4(f), b = load_once_u4(f + 4);
    const uint32_t q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(q[j]);
  } else {
    unpack8(load_once_u4(static_cast<const uint16_t*>(p) + i), v);
  }
}

template <bool F32>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// ---------------------------------------------------------------- stores
// A store past the caches or an ordinary one, by a wave-uniform flag.  The empty
// statements keep the compiler from making one (ordinary) store of both.
template <typename T>
__device__ __forceinline__ void put(T* p, const T& v, int stream) {
  if (stream) {
    asm volatile("");
    __builtin_nontemporal_store(v, p);
    asm volatile("");
  } else {
    *p = v;
  }
}

// An output that cannot stay in the 256 MB Infinity Cache for its reader goes
// past it (the plain product's rule).
inline bool streams(int64_t rows, int64_t row_bytes) { return row_bytes > 0 && rows > ((int64_t)192 << 20) / row_bytes; }

// ---------------------------------------------------------------- E4M3 codes
// Upward exponent for E4M3 (largest magnitude 448 = 1.75 * 2^8) of a finite
// maximum given as fp32 bits: smallest e >= -127 with amax <= 448 * 2^e.
__device__ __forceinline__ int upward_exp_e4m3(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

typedef short s16x2_t __attribute__((ext_vector_type(2)));

// Eight bf16 values -> eight E4M3 bytes of value / 2^e (round to nearest even;
// the upward exponent leaves nothing to saturate).
__device__ __forceinline__ uint2 e4m3_8(const uint4 w, float scale) {
  s16x2_t lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_t, w.x), scale, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_t, w.y), scale, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_t, w.z), scale, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_t, w.w), scale, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

}  // namespace mx
