"""Pins of the norm and dropout oracle: the mask's statistics and layout, the
E4M3 scale rule and codes against torch's float8 conversion, and the norm's
gradients against central differences of its forward formula in float64."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import norm as N
from oracle import philox as P
from oracle import quant as Q


def test_keep_mask_layout():
    rows, cols, seed, offset = 3, 19, 2 ** 40 + 5, 2 ** 33 + 1
    got = N.keep_mask(rows, cols, 0.3, seed, offset)
    thr = int(0.3 * 65536 + 0.5)
    for r in range(rows):
        for c in range(cols):
            i = r * 24 + c
            blk = i >> 3
            w = P.philox4x32_10(blk, 0, offset & 0xFFFFFFFF, offset >> 32, seed & 0xFFFFFFFF, seed >> 32)
            word = int(w[(i >> 1) & 3])
            half = word >> 16 if i & 1 else word & 0xFFFF
            assert got[r, c] == (half >= thr)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 0.1, 0.25, 0.5, 0.9, 1.0])
def test_keep_mask_rate_and_scale(p):
    n = 1 << 18
    keep = N.keep_mask(1, n, p, 7, 3)
    q = 1 - N.threshold(p) / 65536
    # binomial: six standard deviations
    assert abs(keep.mean() - q) <= 6 * np.sqrt(max(q * (1 - q), 0) / n)
    assert float(N.keep_scale(p)) == (np.float32(1 / q) if q > 0 else 0.0)
    if p in (0.0,):
        assert keep.all()
    if p == 1.0:
        assert not keep.any()


def test_masks_of_distinct_offsets_are_independent():
    a, b = (N.keep_mask(64, 4096, 0.5, 7, o) for o in (1, 2))
    n = a.size
    assert abs((a == b).mean() - 0.5) <= 6 * 0.5 / np.sqrt(n)


def test_e4m3_matches_torch_and_the_upward_rule():
    bits = np.arange(0, 0x7F80, dtype=np.uint16)[: 32 * (0x7F80 // 32)]
    rng = np.random.default_rng(1)
    for y in (bits.reshape(1, -1), rng.permutation(bits).reshape(1, -1) ^ np.uint16(0x8000)):
        codes, scales = N.encode_e4m3(y)
        v = F.bf16_bits_to_f64(y).reshape(-1, 32)
        e = scales.reshape(-1).astype(np.int64) - 127
        amax = np.abs(v).max(axis=1)
        assert (amax <= 448 * np.ldexp(1.0, e)).all()
        assert ((e == -127) | (amax > 448 * np.ldexp(1.0, e - 1))).all()
        q = torch.from_numpy(v * np.ldexp(1.0, -e)[:, None])
        # exact in fp32: bf16 values over a power of two, subnormal bits apart
        want = q.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes.reshape(-1, 32), want)
        err = np.abs(N.decode_e4m3(codes, scales).reshape(-1, 32) - v)
        # half a step: 2^-4 of the value, and 2^-10 of the scale below the normal range
        assert (err <= np.maximum(2.0 ** -4 * np.abs(v), np.ldexp(1.0, e - 10)[:, None])).all()


def test_zero_block_takes_the_lowest_scale():
    codes, scales = N.encode_e4m3(np.zeros((2, 64), np.uint16))
    assert (codes == 0).all() and (scales == 0).all()


@pytest.mark.parametrize("t,d", [(1, 32), (3, 64), (5, 96)])
def test_gradients_against_differences(t, d):
    rng = np.random.default_rng(t * 100 + d)
    s, gamma = rng.standard_normal((t, d)), 1 + 0.1 * rng.standard_normal(d)
    dy, ds = rng.standard_normal((t, d)), rng.standard_normal((t, d))
    eps = 1e-2

    def loss(s_, gamma_):
        return float((dy * N.rmsnorm(s_, gamma_, eps)[1]).sum() + (ds * s_).sum())

    rstd, _ = N.rmsnorm(s, gamma, eps)
    got_s, got_g = N.rmsnorm_backward(dy, s, rstd, gamma, ds)
    h = 1e-5
    for _ in range(8):
        u, v = rng.standard_normal((t, d)), rng.standard_normal(d)
        diff = (loss(s + h * u, gamma) - loss(s - h * u, gamma)) / (2 * h)
        # truncation h^2 times a third derivative of order one per element, and rounding 2^-53 / h
        assert abs(diff - (got_s * u).sum()) <= 1e-6 * np.abs(got_s * u).sum()
        diff = (loss(s, gamma + h * v) - loss(s, gamma - h * v)) / (2 * h)
        assert abs(diff - (got_g * v).sum()) <= 1e-6 * np.abs(got_g * v).sum()


def test_dropout_is_its_own_adjoint():
    rng = np.random.default_rng(4)
    x, y = (F.f32_to_f64(rng.standard_normal((5, 37))) for _ in range(2))
    keep, scale = N.keep_mask(5, 37, 0.4, 9, 2), float(N.keep_scale(0.4))
    assert np.isclose(((keep * x * scale) * y).sum(), (x * (keep * y * scale)).sum(), rtol=1e-12)
    bits = N.dropout_bits(x.astype(np.float32), 0.4, 9, 2)
    assert ((F.bf16_bits_to_f64(bits) != 0) == keep).all()


def test_dropout_leaves_no_trace_of_masked_values():
    x = np.ones((4, 40), np.float32)
    keep = N.keep_mask(4, 40, 0.5, 1, 1)
    x[~keep] = np.where(np.arange((~keep).sum()) % 2, np.inf, np.nan)
    out = F.bf16_bits_to_f64(N.dropout_bits(x, 0.5, 1, 1))
    assert np.isfinite(out).all() and (out[~keep] == 0).all() and (out[keep] == 2).all()


def test_e2m1_codes_of_the_norm_are_those_of_the_row_quantizer():
    rng = np.random.default_rng(2)
    s = rng.standard_normal((4, 64))
    y = N.f32_to_bf16_rne(N.rmsnorm(s, np.ones(64), 1e-5)[1].astype(np.float32))
    codes, scales = Q.quantize_rows(y)
    assert codes.shape == (4, 32) and scales.shape == (4, 2)
