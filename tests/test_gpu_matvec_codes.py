"""E4M3 activations of the few-row products over every code and scale byte."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import norm as N
from oracle import nvfp4 as NV


def rounded(v):
    """What a decoded value goes to: the nearest multiple of 2^-133, ties to
    even (exact but under scale bytes 0 to 2), an infinity from 2^128 on."""
    with np.errstate(invalid="ignore"):
        return np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), np.ldexp(np.rint(np.ldexp(v, 133)), -133))


def e4m3_values():
    v = np.append(NV.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64), np.nan)
    return np.concatenate([v, -v])


def test_decoded_codes_of_the_producer_are_exact_in_bf16():
    """Codes of every block maximum with every bf16 magnitude below it, sampled:
    the decoded value is a bf16 value, or 2^128 where the largest one rounds up."""
    rng = np.random.default_rng(1)
    pos = np.arange(0, 0x7F80, dtype=np.uint16)
    for _ in range(8):
        top = rng.permutation(pos)[:, None]
        rest = (rng.random((len(pos), 31)) * (top + 1)).astype(np.uint16)
        near = np.maximum(top.astype(np.int64) - rng.integers(0, 1400, rest.shape), 0).astype(np.uint16)
        y = np.concatenate([top, np.where(rng.random(rest.shape) < 0.5, rest, near)], axis=1)
        v = N.decode_e4m3(*N.encode_e4m3(y))
        fits = np.abs(v) < 2.0 ** 128
        assert (v[~fits] == 2.0 ** 128).all() and (F.bf16_bits_to_f64(y)[~fits] >= 248 * 2.0 ** 120).all()
        back = F.bf16_bits_to_f64(N.f32_to_bf16_rne(np.where(fits, v, 0).astype(np.float32)))
        assert np.array_equal(back, np.where(fits, v, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [16, 64])
def test_every_code_under_every_scale_byte(gpu_lib, m):
    """Rows with one code each against unit weights give that code's value."""
    w = np.zeros((32, 16), np.uint8)
    w[np.arange(32), np.arange(32) // 2] = 2 << (4 * (np.arange(32) % 2))      # 1.0 at column i of row i
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    w, ws = dev(w), torch.full((32, 1), 127, dtype=torch.uint8, device="cuda")
    at = np.arange(m) % 32
    rows = []
    for a in range(0, 256, m):
        x = np.zeros((m, 32), np.uint8)
        x[np.arange(m), at] = np.arange(a, a + m)
        rows.append(dev(x))
    atd = dev(at)[:, None]
    got = torch.stack([torch.cat([gpu_lib.fp4_matvec(x, w, ws, x_scales=torch.full((m, 1), byte, dtype=torch.uint8, device="cuda"))
                                  .gather(1, atd)[:, 0] for x in rows]) for byte in range(255)])
    got = got.cpu().numpy().astype(np.float64)
    values = e4m3_values()[None] * np.ldexp(1.0, np.arange(255) - 127)[:, None]
    want = rounded(values)
    assert np.array_equal(want[3:247], values[3:247], equal_nan=True) and not np.isinf(want[:247]).any()
    assert np.array_equal(got, want, equal_nan=True)
