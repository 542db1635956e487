"""Products of so many tiles that their workgroups take a second launch dimension:
rows and columns on both sides of its shares against the same call on a part, whose
sums are the same in the same order.  Each test needs 10 to 80 GB of device memory
and skips where that is not free."""

import pytest
import torch

from test_gpu_experts_huge import codes, need, release_memory  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def offsets(sizes):
    return torch.tensor([0, *sizes], device="cuda").cumsum(0).int()


def test_rows_of_many_experts(gpu_lib):
    """1024 experts, a row each, against 2^20 weight rows of 32 values: 17 M tiles of 64 x 64."""
    need(40)
    e, n, k = 1024, 1 << 20, 32
    a, b = codes((e, k), 1), codes((e, n, k), 2)
    c = torch.full((e, n), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp4_gemm_experts(offsets([1] * e), *a, *b, c=c)
    one = offsets([1])
    for r in range(0, e, 31):
        want = gpu_lib.fp4_gemm_experts(one, *[v[r:r + 1].clone() for v in a], *[v[r:r + 1] for v in b], dtype=torch.bfloat16)
        assert torch.equal(c[r], want[0]), r
    assert not (c == 7).all(1).any()


def test_product_of_many_columns(gpu_lib):
    """One row against 2^30 + 544 weight rows: 2^22 + 3 tiles of 256 x 256."""
    need(30)
    n, k = (1 << 30) + 544, 32
    a, b = codes((1, k), 1), codes((n, k), 2)
    y = torch.full((1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp4_gemm_act(*a, *b, gpu_lib.FP4_ACT_SILU, y=y)
    half = (1 << 29) + 1024
    for lo in (0, half - 4096, half, (1 << 30) - 8192, n - 4096):
        part = [v[lo:lo + 4096].clone() for v in b]
        assert torch.equal(gpu_lib.fp4_gemm_act(*a, *part, gpu_lib.FP4_ACT_SILU)[0], y[:, lo:lo + 4096]), lo
    assert not any((y[0, i:i + 256] == 7).all() for i in range(0, n, 256 * 9973))


def test_gradients_of_many_experts(gpu_lib):
    """1024 experts' 32 x (2^20 + 256): 4097 tiles each."""
    need(80)
    e, m, n = 1024, 32, (1 << 20) + 256
    a, b = codes((m, 32 * e), 1), codes((n, 32 * e), 2)
    c = torch.full((e, m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp4_gemm_experts_wgrad(offsets([32] * e), *a, *b, c=c)
    for i in (0, 1, 511, 512, 513, 700, 1022, 1023):
        at, sc = slice(16 * i, 16 * i + 16), slice(i, i + 1)
        for lo in (0, n // 2 // 32 * 32, n - 256):
            part = [torch.zeros((r, w), dtype=torch.uint8, device="cuda") for r in (m, 256) for w in (128, 8)]
            part[0][:, :16], part[1][:, :1] = a[0][:, at], a[1][:, sc]
            part[2][:, :16], part[3][:, :1] = b[0][lo:lo + 256, at], b[1][lo:lo + 256, sc]
            want = gpu_lib.fp4_gemm_experts_wgrad(offsets([32]), *part, dtype=torch.bfloat16)
            assert torch.equal(c[i, :, lo:lo + 256], want[0]), (i, lo)


def test_gated_producer_of_many_experts(gpu_lib):
    """32 of 1024 experts with 32 rows each, 2^19 columns: 1028 x 4096 tiles."""
    need(40)
    e, rows, f, d = 1024, 1024, 1 << 19, 32
    x, w = codes((rows, d), 1), codes((e, 2 * f, d), 2)
    busy = set(range(5, e, 32))
    got = gpu_lib.fp4_swiglu_producer_experts(offsets([32 if i in busy else 0 for i in range(e)]), *x, *w, 0x5A5A)
    for r, i in enumerate(sorted(busy)):
        if r % 5 and r != 31:
            continue
        at = slice(32 * r, 32 * r + 32)
        want = gpu_lib.fp4_swiglu_producer_experts(offsets([32]), *[v[at].clone() for v in x], *[v[i:i + 1] for v in w], 0x5A5A)
        assert all(torch.equal(g[at], v) for g, v in zip(got[:4], want[:4])), i
        assert torch.equal(got[4][:, 16 * r:16 * r + 16], want[4]) and torch.equal(got[5][:, r:r + 1], want[5]), i
