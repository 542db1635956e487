// Epilogue of the SwiGLU producers on the fast main loop's tile: a and b in
// bf16, and h = SiLU(a) b as MXFP4 codes, row-facing and column-facing.
#pragma once

#include "gemm_core.h"
#include "mx_device.h"

namespace mx {

// RTN MXFP4 of one 32-value bf16 block given as 16 packed words.
__device__ __forceinline__ uint4 encode_block_bf16(const uint32_t (&w)[16], int& e_out) {
  // largest 15-bit magnitude pattern: packed 16-bit maxima, one final pair
  u16x2_t mm = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j) mm = __builtin_elementwise_max(mm, __builtin_bit_cast(u16x2_t, w[j] & 0x7FFF7FFFu));
  const uint32_t m = max((uint32_t)mm[0], (uint32_t)mm[1]);
  const int e = upward_exp(m << 16);
  const float sc = pow2_scale(e);
  e_out = e;
  return make_uint4(rtn8_bf16(w[0], w[1], w[2], w[3], sc), rtn8_bf16(w[4], w[5], w[6], w[7], sc),
                    rtn8_bf16(w[8], w[9], w[10], w[11], sc), rtn8_bf16(w[12], w[13], w[14], w[15], sc));
}

// SwiGLU producer epilogue for the 8-wave tile (256 tokens x 128 FFN columns;
// wave (wm, wn) holds a in sub-tile 0 and b in sub-tile 1 for FFN columns
// wn*32 ..).  LDS (free after the main loop) holds two staged bf16 tiles of
// 256 rows x kHPitch bytes: h in the first, a then b in the second.  Within a
// row, dword d sits at d ^ hswz(row) so that the column-pair reads of the H32
// pass (8 lanes per column pair, one per token block) hit distinct banks; the
// XOR moves whole 8-dword groups, so 16-byte chunks stay contiguous.
//   pass 1  a, b, h in bf16 (a and b are the rounded GEMM outputs)
//   pass 2  a out with whole-row stores; h row codes (4 lanes per row: 64
//           contiguous bytes); h column codes with H32 (8 lanes per column:
//           one whole 128-byte line)
//   pass 3  b through the same buffer as a
// Rows T and beyond are not written; a column of h codes holds ldt tokens.
__device__ __forceinline__ int hswz(int row) { return ((row >> 5) & 7) << 3; }

__device__ __forceinline__ void swiglu_epilogue_staged(
    uint8_t* smem, const v16f (&acc)[4][2], int64_t T, int64_t ldt, int64_t Fdim, int64_t m0, int64_t n0, int wave, int lane,
    int wm, int wn, int hl, uint16_t* __restrict__ a_out, uint16_t* __restrict__ b_out,
    uint8_t* __restrict__ h_codes, uint8_t* __restrict__ h_scales, uint8_t* __restrict__ ht_codes,
    uint8_t* __restrict__ ht_scales, uint32_t sign_mask16) {
  uint8_t* hs = smem;
  uint8_t* as = smem + 256 * kHPitch;
  const int tid = threadIdx.x;
  uint32_t bpk[4][4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = wm * 128 + 32 * i + (lane & 31);
    // a and b of the lane's 16 columns of row lr in bf16, then SiLU of all 16
    // in one batch
    uint32_t ab[4][2], bb[4][2];
    float av[16], sg[16], sl[16];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ab[g][u] = bf16_pack2_rne(acc[i][0][4 * g + 2 * u], acc[i][0][4 * g + 2 * u + 1]);
        bb[g][u] = bf16_pack2_rne(acc[i][1][4 * g + 2 * u], acc[i][1][4 * g + 2 * u + 1]);
        av[4 * g + 2 * u] = __uint_as_float(ab[g][u] << 16);
        av[4 * g + 2 * u + 1] = __uint_as_float(ab[g][u] & 0xFFFF0000u);
      }
    sigmoid_silu_n<16>(av, sg, sl);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int dw = (wn * 32 + 8 * g + 4 * hl) >> 1;     // first dword of the lane's 4 columns
      uint32_t hb[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        hb[u] = bf16_pack2_rne(__fmul_rn(sl[4 * g + 2 * u], __uint_as_float(bb[g][u] << 16)),
                               __fmul_rn(sl[4 * g + 2 * u + 1], __uint_as_float(bb[g][u] & 0xFFFF0000u)));
      const int off = lr * kHPitch + 4 * (dw ^ hswz(lr));
      *reinterpret_cast<uint2*>(hs + off) = make_uint2(hb[0], hb[1]);
      *reinterpret_cast<uint2*>(as + off) = make_uint2(ab[g][0], ab[g][1]);
      bpk[i][g][0] = bb[g][0];
      bpk[i][g][1] = bb[g][1];
    }
  }
  __syncthreads();
  // a out: 16 lanes per row (256 bytes), 32 rows per pass of the workgroup
  const int ch = tid & 15;
#pragma unroll 4
  for (int p = 0; p < 8; ++p) {
    const int r = 32 * p + (tid >> 4);
    const int64_t row = m0 + r, col = n0 + 8 * ch;
    if (row < T && col < Fdim)
      __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(as + r * kHPitch + 4 * ((4 * ch) ^ hswz(r))),
                                  reinterpret_cast<v4i*>(a_out + row * Fdim + col));
  }
  // h row codes: thread (row b/4, block b%4)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int b = tid + 512 * k, lr = b >> 2, blk = b & 3;
    const int64_t row = m0 + lr, col0 = n0 + 32 * blk;
    uint32_t wv[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 d = *reinterpret_cast<const uint4*>(hs + lr * kHPitch + 4 * ((16 * blk + 4 * q) ^ hswz(lr)));
      wv[4 * q] = d.x; wv[4 * q + 1] = d.y; wv[4 * q + 2] = d.z; wv[4 * q + 3] = d.w;
    }
    int e;
    const uint4 code = encode_block_bf16(wv, e);
    if (row < T && col0 < Fdim) {
      *reinterpret_cast<uint4*>(h_codes + row * (Fdim >> 1) + (col0 >> 1)) = code;
      h_scales[row * (Fdim >> 5) + (col0 >> 5)] = (uint8_t)(e + 127);
    }
  }
  // h column codes with H32: thread (column pair tid/8, token block tid%8)
  if (ht_codes != nullptr) {
    const int cp = tid >> 3, tb = tid & 7;
    const int64_t r0 = m0 + 32 * tb;
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = *reinterpret_cast<const uint32_t*>(hs + (32 * tb + i) * kHPitch + 4 * (cp ^ (tb << 3)));
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int64_t col = n0 + 2 * cp + c;
      float fv[32];
      h32_column(v, c, sign_mask16, fv);
      h32_fp32(fv);
      int e;
      const uint4 code = encode32_rtn(fv, e);
      if (r0 < T && col < Fdim) {
        __builtin_nontemporal_store(v4i{(int)code.x, (int)code.y, (int)code.z, (int)code.w},
                                    reinterpret_cast<v4i*>(ht_codes + col * (ldt >> 1) + (r0 >> 1)));
        ht_scales[col * (ldt >> 5) + (r0 >> 5)] = (uint8_t)(e + 127);
      }
    }
  }
  __syncthreads();
  // b through the a buffer
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lr = wm * 128 + 32 * i + (lane & 31);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int dw = (wn * 32 + 8 * g + 4 * hl) >> 1;
      *reinterpret_cast<uint2*>(as + lr * kHPitch + 4 * (dw ^ hswz(lr))) = make_uint2(bpk[i][g][0], bpk[i][g][1]);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int p = 0; p < 8; ++p) {
    const int r = 32 * p + (tid >> 4);
    const int64_t row = m0 + r, col = n0 + 8 * ch;
    if (row < T && col < Fdim)
      __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(as + r * kHPitch + 4 * ((4 * ch) ^ hswz(r))),
                                  reinterpret_cast<v4i*>(b_out + row * Fdim + col));
  }
}

}  // namespace mx
