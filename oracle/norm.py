"""Dropout, the residual RMSNorm boundary with its codes, and its gradients (oracle).

"Format-Aware Fusion for Fast FP4 Pretraining", §3.1-§3.2: a producer in front
of a quantized linear layer keeps the bf16 residual and the row statistics and
emits the codes its consumer reads; §2.2.1: block scales are rounded upward;
App. A.1: random state is a seed plus a counter offset.

Readings (the pages print no norm):
  * dropout: element c of row r has index i = r * 8 ceil(cols / 8) + c and
    takes half i & 1 (0: low) of word (i >> 1) & 3 of the Philox block at
    counter (i >> 3, offset); it is kept iff the half is >= thr,
    thr = floor(65536 p + 1/2), and scaled by RN32(65536 / (65536 - thr));
  * s = bf16(fp32 sum), the kept element and the residual in one fused
    multiply-add; the norm is taken of the rounded s;
  * y = bf16(s rstd gamma), rstd = 1 / sqrt(mean(s^2) + eps);
  * E4M3 codes: 32 values under 2^e, e the smallest integer >= -127 with
    amax <= 448 * 2^e, nearest even; E2M1 codes: quantize_rows of y.
The mask, s and the codes of a given y are exact; rstd, y and the gradients are
float64 values of the formulas, which the kernels meet within fp32 rounding.
"""

import numpy as np

from . import formats as F
from . import nvfp4 as NV
from . import philox as P
from .swiglu import f32_to_bf16_rne, fma_f32

E4M3_MAX = 448.0


def threshold(p):
    """thr of a probability given as fp32 (what the C call receives)."""
    return int(np.floor(np.float64(np.float32(p)) * 65536.0 + 0.5))


def keep_scale(p):
    thr = threshold(p)
    return np.float32(65536.0 / (65536.0 - thr)) if thr < 65536 else np.float32(0.0)


def keep_mask(rows, cols, p, seed, offset):
    """Boolean [rows][cols]."""
    pitch = 8 * ((cols + 7) // 8)
    i = (np.arange(rows, dtype=np.uint64)[:, None] * np.uint64(pitch) + np.arange(cols, dtype=np.uint64)[None, :])
    word = P.draws(seed, offset, ((i >> np.uint64(3)) << np.uint64(2)) + ((i >> np.uint64(1)) & np.uint64(3)))
    half = np.where(i & np.uint64(1), word >> np.uint64(16), word & np.uint64(0xFFFF))
    return half >= np.uint64(threshold(p))


def dropout_bits(x_f32, p, seed=0, offset=0, residual_bits=None):
    """bf16 bits of fp32 x [rows][cols] after dropout and the residual's addition."""
    x = np.asarray(x_f32, dtype=np.float32)
    keep, scale = keep_mask(*x.shape, p, seed, offset), keep_scale(p)
    with np.errstate(invalid="ignore", over="ignore"):
        if residual_bits is None:
            return f32_to_bf16_rne(np.where(keep, x * scale, np.float32(0.0)))
        res = F.bf16_bits_to_f64(residual_bits).astype(np.float32)
        return f32_to_bf16_rne(np.where(keep, fma_f32(x, np.broadcast_to(scale, x.shape), res), res))


def upward_exponent_e4m3(amax):
    """Smallest integer e >= -127 with amax <= 448 * 2**e."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127, dtype=np.int64)
    for _ in range(260):
        e = np.where(amax > E4M3_MAX * np.ldexp(1.0, e), e + 1, e)
    return e


def encode_e4m3(y_bits):
    """(codes [t][d], scales [t][d/32]) of bf16 bits."""
    y = F.bf16_bits_to_f64(y_bits)
    t, d = y.shape
    b = y.reshape(t, d // 32, 32)
    e = upward_exponent_e4m3(np.abs(b).max(axis=-1))
    mag = np.abs(b) * np.ldexp(1.0, -e)[..., None]
    code = NV.e4m3_round(mag)[0].astype(np.uint8) | (np.signbit(b).astype(np.uint8) << 7)
    return code.reshape(t, d).astype(np.uint8), (e + 127).astype(np.uint8)


def decode_e4m3(codes, scales):
    codes = np.asarray(codes, dtype=np.uint8)
    v = NV.e4m3_decode(codes & 0x7F)
    v = np.where(codes & 0x80, -v, v)
    t, d = codes.shape
    s = np.ldexp(1.0, np.asarray(scales, dtype=np.int64) - 127)
    return (v.reshape(t, d // 32, 32) * s[..., None]).reshape(t, d)


def rmsnorm(s64, gamma64, eps):
    """(rstd [t], y [t][d]) in float64."""
    rstd = 1.0 / np.sqrt(np.mean(s64 * s64, axis=-1) + np.float64(np.float32(eps)))
    return rstd, s64 * rstd[:, None] * gamma64


def rmsnorm_backward(dy64, s64, rstd64, gamma64, ds64=None):
    """(ds', dgamma) in float64, with the statistic rstd as given."""
    xh, g = s64 * rstd64[:, None], dy64 * gamma64
    ds = rstd64[:, None] * (g - xh * np.mean(g * xh, axis=-1, keepdims=True))
    return ds if ds64 is None else ds + ds64, (dy64 * xh).sum(axis=0)
