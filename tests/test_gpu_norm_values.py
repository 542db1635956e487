"""The norm producer's values at the ends of their ranges."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import formats as F
from oracle import norm as N

pytestmark = pytest.mark.gpu


def dev16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def val(t):
    return F.bf16_bits_to_f64(host(t.contiguous().view(torch.int16)).view(np.uint16))


SHAPES = [(3, 96), (2, 544), (2, 2080), (1, 8224), (1, 32768)]


def check_past_the_range(mx, s_bits, g):
    """y against float64 rounded once: from 2^128 - 2^119 on (half a bf16 step
    past the largest bf16 value) an infinity with the product's sign."""
    s, g_bits = F.bf16_bits_to_f64(s_bits), synthetic.bf16_bits(g)
    y = val(mx.fp4_rmsnorm_producer(dev16(s_bits), dev16(g_bits), emit_y=True)[2])
    with np.errstate(invalid="ignore", over="ignore"):
        want = N.rmsnorm(s, F.bf16_bits_to_f64(g_bits), 1e-5)[1]
        top = 2.0 ** 128 - 2.0 ** 119
        # one fp32 rounding on either side of the border may go either way
        sure = ~(np.abs(np.abs(want) - top) <= 2.0 ** 104)
        want = np.where(np.abs(want) >= top, np.copysign(np.inf, want), want)
    assert sure.mean() > 0.99 and np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want) & sure
    assert np.array_equal(y[inf], want[inf])
    fin = np.isfinite(want) & sure
    # a bf16 rounding, and one of fp32 before it
    assert (np.abs(y[fin] - want[fin]) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want[fin]) + 2.0 ** -133).all()
    return want, inf


@pytest.mark.parametrize("t,d", SHAPES)
def test_infinite_and_nan_gamma_stay_in_their_columns(gpu_lib, t, d):
    s_bits = synthetic.tensor((t, d), seed=51)
    s_bits[:, 5] = 0
    g = np.ones(d, np.float32)
    g[0:4] = [2.0 ** 127, -2.0 ** 127, 2.0 ** 126, 1.5 * 2.0 ** 127]
    g[4:9] = [np.inf, np.inf, -np.inf, np.nan, 2.0 ** -126]
    g[16:32] = 2.0 ** np.arange(112, 128)
    s_bits[np.abs(F.bf16_bits_to_f64(s_bits)) < 2.0 ** -6] = 0x3F80   # away from zero, but for column 5
    s_bits[:, 5] = 0
    want, inf = check_past_the_range(gpu_lib, s_bits, g)
    # 0 times an infinity is NaN
    assert inf[:, [4, 6]].all() and np.isnan(want[:, [5, 7]]).all()


@pytest.mark.parametrize("t,d", SHAPES)
def test_products_past_the_range_are_infinities(gpu_lib, t, d):
    s_bits = synthetic.tensor((t, d), std=1.0, seed=52, outlier_rate=0.002, outlier_scale=20.0)
    rng = np.random.default_rng(53)
    g = (rng.choice([-1.0, 1.0], d) * rng.uniform(1, 1.99, d) * 2.0 ** rng.integers(124, 128, d)).astype(np.float32)
    want, inf = check_past_the_range(gpu_lib, s_bits, g)
    assert 0.01 < inf.mean() < 0.5 and (want[inf] > 0).any() and (want[inf] < 0).any()


@pytest.mark.parametrize("t,d", [(40, 32), (9, 160), (7, 2048), (3, 4096), (3, 32768)])
def test_non_finite_rows_stay_apart(gpu_lib, t, d):
    """A row with an infinity or NaN becomes NaN, rows beside it (of the same
    wave too) keep their bytes, forwards and backwards."""
    mx = gpu_lib
    s = dev16(synthetic.tensor((t, d), std=1.0, seed=54))
    dy = dev16(synthetic.tensor((t, d), std=1.0, seed=55))
    g = torch.linspace(0.5, 1.5, d, device="cuda").bfloat16()
    clean = mx.fp4_rmsnorm_producer(s, g, emit_y=True)
    grad = mx.fp4_rmsnorm_backward(dy, s, clean[1], g, ds=dy)
    bad, bad_dy = s.clone(), dy.clone()
    rows = [1] if t == 3 else [1, 4, t - 1]
    for r, v in zip(rows, (float("inf"), float("nan"), -float("inf"))):
        bad[r, (7 * r) % d] = v
        bad_dy[r, (5 * r + 1) % d] = v
    rest = [r for r in range(t) if r not in rows]
    got = mx.fp4_rmsnorm_producer(bad, g, emit_y=True)
    for k, (a, b) in enumerate(zip(got, clean)):
        assert torch.equal(a[rest], b[rest]), k
    assert got[1][rows].isnan().all() and got[2][rows].isnan().all()
    for first, second, rstd in ((dy, bad, got[1]), (bad_dy, s, clean[1])):
        dsum, _, dgamma = mx.fp4_rmsnorm_backward(first, second, rstd, g, ds=dy)
        assert torch.equal(dsum[rest], grad[0][rest]) and not dsum[rows].isfinite().all(1).any()
        # every column of a row whose rstd is NaN, else only the columns of the infinities and NaN
        assert dgamma.isnan().all() if second is bad else (~dgamma.isfinite()).sum() == len(rows)


U, H = 2.0 ** -24, 2.0 ** -8                             # half an fp32 step, half a bf16 step
WIDTHS = [32, 160, 544, 1056, 2048, 2080, 4128, 8192, 8224, 16416, 32768]


@pytest.mark.parametrize("d", WIDTHS)
def test_the_statistic_is_held_in_64_bits(gpu_lib, d):
    """Small integers: a thread's sum of at most 32 squares of up to 255 is exact
    in fp32, so that what remains is 64-bit work, one rounding to fp32 of rstd
    (2^-40 stands for the 64-bit roundings), and for y one fp32 rounding before
    bf16's: y is the float64 value rounded once wherever no tie lies within that
    rounding.  A statistic in fp32 steps, or y in three, is further off."""
    mx, rng = gpu_lib, np.random.default_rng(d)
    t = max(3, (1 << 19) // d)
    s = rng.integers(-255, 256, (t, d)).astype(np.float32)
    s[0] = rng.integers(1, 4, d)
    g_bits = synthetic.bf16_bits((1 + 0.3 * rng.standard_normal(d)).astype(np.float32))
    eps = 1e-5
    got = mx.fp4_rmsnorm_producer(dev16(synthetic.bf16_bits(s)), dev16(g_bits), eps, emit_y=True)
    r64, y64 = N.rmsnorm(s.astype(np.float64), F.bf16_bits_to_f64(g_bits), eps)
    assert (np.abs(host(got[1]).astype(np.float64) - r64) <= (U + 2.0 ** -40) * r64).all()
    size = np.abs(y64)
    step = 2.0 ** (np.floor(np.log2(np.where(size > 0, size, 1.0))) - 7)
    low = np.floor(size / step) * step                   # the bf16 value below
    tie = np.abs(size - (low + step / 2)) <= (U + 2.0 ** -36) * size
    want = np.copysign(np.where(size - low > step / 2, low + step, low), y64)
    y = val(got[2])
    assert tie.mean() < 2.0 ** -12
    assert np.array_equal(y[~tie], want[~tie])
    assert (np.abs(y - y64) <= (H + 2 * U) * size).all()


@pytest.mark.parametrize("d", WIDTHS)
def test_the_statistic_of_any_row(gpu_lib, d):
    """Squares that round: at most 32 fused steps of a thread on a sum of
    positive terms, of which the root halves the error, and rstd's rounding."""
    s_bits = synthetic.tensor((5, d), std=1.0, seed=56, outlier_rate=0.002, outlier_scale=20.0)
    got = gpu_lib.fp4_rmsnorm_producer(dev16(s_bits), dev16(synthetic.bf16_bits(np.ones(d, np.float32))), emit_codes=False)
    r64 = N.rmsnorm(F.bf16_bits_to_f64(s_bits), np.ones(d), 1e-5)[0]
    assert (np.abs(host(got[1]).astype(np.float64) - r64) <= 17.5 * U * r64).all()
