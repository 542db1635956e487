"""The norm calls over many rows: more rows than a launch's first dimension
holds, offsets past 32 bits."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import formats as F
from oracle import norm as N
from oracle import philox as P
from oracle import quant as Q

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
