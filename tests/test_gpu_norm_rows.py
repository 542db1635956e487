"""The norm calls over many rows: more rows than a launch's first dimension
holds, offsets past 32 bits."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import norm as N
from oracle import philox as P

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8                             # half an fp32 step, half a bf16 step
TINY = 2.0 ** -133                                       # the subnormal bf16 spacing


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def val(t):
    return F.bf16_bits_to_f64(bits(t))


def row_mask(r, cols, p, seed, offset):
    """The kept elements of one row."""
    i = np.uint64(r) * np.uint64(8 * -(-cols // 8)) + np.arange(cols, dtype=np.uint64)
    word = P.draws(seed, offset, ((i >> np.uint64(3)) << np.uint64(2)) + ((i >> np.uint64(1)) & np.uint64(3)))
    return np.where(i & np.uint64(1), word >> np.uint64(16), word & np.uint64(0xFFFF)) >= N.threshold(p)


@pytest.fixture
def room():
    """Free device memory, given back after the test."""
    torch.cuda.empty_cache()
    yield torch.cuda.mem_get_info()[0]
    torch.cuda.empty_cache()


# 2^32 threads and a few rows more, at sixteen, four and one row a workgroup
@pytest.mark.parametrize("t,d", [((1 << 28) + 17, 32), ((1 << 26) + 5, 160), ((1 << 24) + 3, 2080)])
def test_more_rows_than_a_launch_dimension_holds(gpu_lib, room, t, d):
    mx = gpu_lib
    if room < 4 * t * d * 2:
        pytest.skip(f"needs {4 * t * d * 2 >> 30} GiB of free device memory")
    x = torch.empty((t, d), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(t))
    gamma = torch.linspace(0.5, 1.5, d, device="cuda").bfloat16()
    s, rstd, _, codes, scales = mx.fp4_rmsnorm_producer(x, gamma, fmt=mx.FP4_E2M1)
    assert torch.equal(s, x)
    for a in range(0, t, t // 5):                        # the same rows by smaller calls
        b = min(t, a + t // 5)
        part = mx.fp4_rmsnorm_producer(x[a:b], gamma, fmt=mx.FP4_E2M1, emit_sum=False)
        for whole, some in ((rstd, part[1]), (codes, part[3]), (scales, part[4])):
            assert torch.equal(whole[a:b], some), a
    # the mask goes by the row's index in the whole tensor
    p, seed, offset = 0.25, 2 ** 40 + 3, 2 ** 33 + 1
    s = mx.fp4_rmsnorm_producer(x, gamma, p=p, seed=seed, offset=offset, emit_codes=False, out=(s, rstd, None, None, None))[0]
    for r in (0, t // 3, t - 20, t - 1):
        want = N.f32_to_bf16_rne(np.where(row_mask(r, d, p, seed, offset), val(x[r:r + 1])[0].astype(np.float32)
                                          * N.keep_scale(p), np.float32(0)))
        assert np.array_equal(bits(s[r:r + 1])[0], want), r


# several turns of a workgroup over its rows, with full and ragged last ones, for
# every number of threads a row and of columns a thread, below and from the
# number of rows on that takes two workgroups a CU
WALKS = [(33000, 32), (40000, 128), (9001, 160), (9001, 544), (5000, 1056), (2500, 1568), (8200, 2048), (2500, 2080),
         (2047, 4096), (2048, 4096), (2100, 4096), (700, 6144), (600, 8192), (520, 8224), (1030, 16384), (515, 32768)]


@pytest.mark.parametrize("t,d", WALKS)
@pytest.mark.parametrize("f32,with_ds,p", [(True, True, 0.1), (False, False, 0.0), (True, False, 0.5), (False, True, 0.0)])
def test_backward_walks_its_rows(gpu_lib, t, d, f32, with_ds, p):
    """With u = 2^-24 and h = 2^-8 (half a bf16 step): dsum as the mean's
    products and its at most 54 sums on mean |g xh| and five more operations,
    then h; dgamma two product roundings and a thread's turns (at most t / 512
    and 8), lanes, waves, at most 16 partial sums a slice and 32 slices on sum
    |dy xh|."""
    mx, g = gpu_lib, torch.Generator("cuda").manual_seed(t + d)
    rand = lambda *n, k=1.0: k * torch.randn(n, device="cuda", generator=g)  # noqa: E731
    s, gamma = rand(t, d, k=2.0).bfloat16(), (1 + 0.2 * rand(d)).bfloat16()
    s[t // 2] = 0                                        # rstd = 1 / sqrt(eps)
    dy = rand(t, d, k=1e-3)
    dy = dy if f32 else dy.bfloat16()
    ds = rand(t, d, k=1e-3).bfloat16() if with_ds else None
    rstd = (s.double().square().mean(1) + 1e-5).rsqrt().float()
    seed, offset = 78, 2 ** 41 + 7
    dsum, dx, dgamma = mx.fp4_rmsnorm_backward(dy, s, rstd, gamma, ds, p, seed, offset)
    r = rstd.double()[:, None]
    xh, gr = s.double() * r, dy.double() * gamma.double()
    want = r * (gr - xh * (gr * xh).mean(1, keepdim=True))
    size = r * (gr.abs() + xh.abs() * (gr * xh).abs().mean(1, keepdim=True))
    if with_ds:
        want, size = want + ds.double(), size + ds.double().abs()
    near = lambda got, ref, m: bool(((got.double() - ref).abs() <= H * ref.abs() + 64 * U * m + TINY).all())  # noqa: E731
    assert near(dsum, want, size)
    terms = dy.double() * xh
    assert ((dgamma.double() - terms.sum(0)).abs() <= (t / 512 + 72) * U * terms.abs().sum(0) + 2.0 ** -149).all()
    if p == 0:
        assert dx is dsum
    else:
        # the mask that dropout alone draws, and dx = 0 under it
        scale = float(N.keep_scale(p))
        keep = mx.fp4_dropout(torch.ones_like(s), p, seed, offset) != 0
        assert (dx[~keep] == 0).all() and near(dx, torch.where(keep, want * scale, 0.0), scale * size)
        for row in (0, t - 1):
            assert np.array_equal(host(keep[row]), row_mask(row, d, p, seed, offset))
    again = mx.fp4_rmsnorm_backward(dy, s, rstd, gamma, ds, p, seed, offset)
    assert torch.equal(again[0], dsum) and torch.equal(again[2], dgamma)


def test_masks_past_2_to_32_blocks(gpu_lib, room):
    """More than 2^32 groups of eight columns: the counter's second word."""
    mx, p, seed, offset = gpu_lib, 0.25, 2 ** 50 + 1, 2 ** 34 + 5
    scale = F.bf16_bits_to_f64(N.f32_to_bf16_rne(N.keep_scale(p)))
    t, d = (1 << 20) + 3, 32768
    size = 2 * t * (d + 8)
    if room < 2.2 * size:
        pytest.skip(f"needs {int(2.2 * size) >> 30} GiB of free device memory")
    x = torch.ones((t, d + 8), dtype=torch.bfloat16, device="cuda")
    assert mx.fp4_dropout(x, p, seed, offset, out=x) is x
    near = (1 << 35) // (d + 8)                           # the row that holds block 2^32
    for r in (0, near - 1, near, near + 1, t - 1):
        assert np.array_equal(val(x[r:r + 1])[0], np.where(row_mask(r, d + 8, p, seed, offset), scale, 0.0)), r
    del x
    x, ones = torch.ones((t, d), dtype=torch.bfloat16, device="cuda"), torch.ones(d, dtype=torch.bfloat16, device="cuda")
    s, rstd, *_ = mx.fp4_rmsnorm_producer(x, ones, p=p, seed=seed, offset=offset, emit_codes=False)
    for r in (0, (1 << 20) - 1, 1 << 20, t - 1):
        assert np.array_equal(val(s[r:r + 1])[0], np.where(row_mask(r, d, p, seed, offset), scale, 0.0)), r
        want = 1 / np.sqrt(np.mean(val(s[r:r + 1])[0] ** 2) + np.float64(np.float32(1e-5)))
        assert abs(float(rstd[r]) - want) <= 17.5 * U * want


def test_backward_past_32_bit_offsets(gpu_lib, room):
    """Rows on both sides of 2^32 elements against calls on those rows alone."""
    mx, p, seed, offset = gpu_lib, 0.3, 3, 2 ** 32 + 7
    t, d = (1 << 21) + 9, 2080
    if room < 6 * t * d * 2:
        pytest.skip(f"needs {6 * t * d * 2 >> 30} GiB of free device memory")
    g = torch.Generator("cuda").manual_seed(9)
    dy, s = (torch.empty((t, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    gamma, rstd = torch.linspace(0.5, 1.5, d, device="cuda").bfloat16(), torch.rand(t, device="cuda", generator=g) + 0.5
    dsum, dx, dgamma = mx.fp4_rmsnorm_backward(dy, s, rstd, gamma, dy, p, seed, offset)
    near = (1 << 32) // d
    total = torch.zeros(d, dtype=torch.float64, device="cuda")
    size = torch.zeros(d, dtype=torch.float64, device="cuda")
    for a in range(0, t, 1 << 16):
        b = min(t, a + (1 << 16))
        part = mx.fp4_rmsnorm_backward(dy[a:b], s[a:b], rstd[a:b], gamma, dy[a:b])
        assert torch.equal(dsum[a:b], part[0]), a
        terms = dy[a:b].double() * (s[a:b].double() * rstd[a:b, None].double())
        total += terms.sum(0)
        size += terms.abs().sum(0)
    assert ((dgamma.double() - total).abs() <= (t / 512 + 72) * U * size).all()
    scale = N.keep_scale(p)
    for r in (0, near - 1, near, near + 1, t - 1):
        keep = row_mask(r, d, p, seed, offset)
        got, want = val(dx[r:r + 1])[0], val(dsum[r:r + 1])[0] * float(scale)
        # dx rounds the unrounded gradient: two half steps from the rounded one's multiple
        assert (got[~keep] == 0).all() and (np.abs(got - want)[keep] <= 2.02 * H * np.abs(want[keep]) + TINY).all(), r
