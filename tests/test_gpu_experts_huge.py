"""The expert and epilogue calls on tensors whose elements pass 2^32: sampled rows
on both sides of the places where a 32-bit index would wrap, against float64.  Each
test needs 20-70 GB of device memory and skips where that is not free."""

import numpy as np
import pytest
import torch

from oracle import act as A
from oracle import formats as F
from oracle import quant as Q

pytestmark = pytest.mark.gpu
GIB, H, U = 1 << 30, 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def release_memory():
    """Hand the cached blocks back after each test, so that the next one's
    free-memory check sees them."""
    yield
    torch.cuda.empty_cache()


def need(gib):
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < gib * GIB:
        pytest.skip(f"needs {gib} GiB of free device memory, {free / GIB:.0f} free")


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()


def samples(rows, cols):
    """Rows around each 2^31 elements, the first and the last."""
    at = {0, 1, rows - 2, rows - 1}
    for p in range(1, rows * cols // (1 << 31) + 1):
        r = p * (1 << 31) // cols
        at |= {r - 1, r, min(r + 1, rows - 1)}
    return sorted(r for r in at if 0 <= r < rows)


D = 4096
T, K = 150_016, 8                                          # 1.2 M rows: 4.9 G elements


def test_tokens_out_and_back(gpu_lib):
    need(60)
    mx = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, D), device="cuda", generator=g).bfloat16()
    ids = torch.rand((T, 16), device="cuda", generator=g).topk(K, -1).indices.int()
    offsets, slots, rows = mx.fp4_expert_sort(ids, 16, 32)
    n = slots.numel()
    assert n * D > 1 << 32
    where = host(rows)
    assert np.array_equal(host(slots)[where.reshape(-1)], np.arange(T * K))
    xs, codes, scales = mx.fp4_expert_gather(x, slots, K)
    at = samples(n, D)
    for r in at:
        s = int(slots[r])
        want = host(x[s // K]) if s >= 0 else np.zeros(D, np.float32)
        assert np.array_equal(host(xs[r]), want)
        wc, ws = Q.quantize_rows((want.view(np.uint32) >> 16).astype(np.uint16)[None])
        assert np.array_equal(host(codes[r])[None], wc) and np.array_equal(host(scales[r])[None], ws)
    del codes, scales
    w = torch.rand((T, K), device="cuda", generator=g)
    y = mx.fp4_expert_combine(xs, rows, w)
    dz, dw = mx.fp4_expert_combine_backward(x, xs, slots, rows, w)
    for t in (0, T // 3, T - 1):
        xt, wt = host(x[t]).astype(np.float64), host(w[t]).astype(np.float64)
        assert (np.abs(host(y[t]) - xt * wt.sum()) <= (H + (K + 1) * U) * np.abs(xt) * wt.sum() + 1e-30).all()
        assert (np.abs(host(dw[t]) - xt @ xt) <= (8 * -(-D // 512) + 7) * U * (xt @ xt)).all()
    for r in at:
        s = int(slots[r])
        want = host(x[s // K]).astype(np.float64) * float(w[s // K, s % K]) if s >= 0 else np.zeros(D)
        assert (np.abs(host(dz[r]) - want) <= (H + 2 * U) * np.abs(want)).all()


def test_act_backward(gpu_lib):
    need(40)
    m, n = 1_100_003, D
    z = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    z.copy_(torch.linspace(-4, 4, n, device="cuda").bfloat16())
    z[m - 1] = 1.5
    dy = torch.ones((m, n), dtype=torch.bfloat16, device="cuda")
    dz, dbias = gpu_lib.fp4_act_backward(dy, z, A.GELU)
    slope = A.slope(host(z[0]), A.GELU)
    for r in samples(m, n):
        want = A.slope(host(z[r]), A.GELU)
        assert (np.abs(host(dz[r]) - want) <= 1e-5 + H * (np.abs(want) + 1e-5)).all()
    # 1.1 M equal terms: fp32 sums of a few thousand, each within its own steps
    assert np.allclose(host(dbias), slope * (m - 1) + A.slope(1.5, A.GELU), rtol=1e-3, atol=m * 1e-5)


def codes(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    *lead, k = shape
    return (torch.randint(0, 256, (*lead, k // 2), dtype=torch.uint8, device="cuda", generator=g),
            torch.randint(118, 124, (*lead, k // 32), dtype=torch.uint8, device="cuda", generator=g))


def value(c, s):
    return F.decode(np.atleast_2d(host(c)), np.atleast_2d(host(s)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_of_many_rows(gpu_lib, dtype):
    need(50)
    m, n, k = 1_060_000, D, 64
    a, b = codes((m, k), 1), codes((2, n, k), 2)
    res = torch.ones((m, n), dtype=torch.bfloat16, device="cuda")
    y, z = gpu_lib.fp4_gemm_act(*a, b[0][0], b[1][0], A.NONE, residual=res, dtype=dtype, emit_z=True)
    at, B = samples(m, n), [value(b[0][i], b[1][i]) for i in range(2)]
    tol = H if dtype is torch.bfloat16 else 0.0
    for r in at:
        A64 = value(a[0][r], a[1][r])
        want, e = (A64 @ B[0].T)[0], (abs(A64) @ abs(B[0]).T)[0]
        assert (np.abs(host(y[r]) - want - 1) <= 1e-5 * e + U * (np.abs(want) + 1) + tol * (np.abs(want + 1) + 1e-5 * e)).all()
        assert (np.abs(host(z[r]) - want) <= 1e-5 * e + H * (np.abs(want) + 1e-5 * e)).all()
    del res, y, z
    split = m - 300_000
    offsets = torch.tensor([0, split, m - 77], dtype=torch.int32, device="cuda")
    c = gpu_lib.fp4_gemm_experts(offsets, *a, *b, dtype=dtype)
    for r in at + [split - 1, split]:
        A64, i = value(a[0][r], a[1][r]), int(r >= split)
        want, e = (A64 @ B[i].T)[0], (abs(A64) @ abs(B[i]).T)[0]
        if r >= m - 77:
            want, e = 0 * want, 0 * e
        assert (np.abs(host(c[r]) - want) <= 1e-5 * e + tol * (np.abs(want) + 1e-5 * e)).all(), r


def test_weight_gradients_of_many_experts(gpu_lib):
    need(40)
    E, m, n = 1000, 2048, 2112                             # 4.3 G elements
    tokens = E * 32 + 256 - E * 32 % 256
    offsets = (torch.arange(E + 1, device="cuda", dtype=torch.int32) * 32)
    a, b = codes((m, tokens), 1), codes((n, tokens), 2)
    c = gpu_lib.fp4_gemm_experts_wgrad(offsets, *a, *b)
    assert c.numel() > 1 << 32
    B = value(*b)
    for e, r in ((0, 0), (496, 1000), (497, 7), (993, 2047), (E - 1, m - 1)):
        left = value(a[0][r], a[1][r])[:, 32 * e:32 * e + 32]
        want, mag = (left @ B[:, 32 * e:32 * e + 32].T)[0], (abs(left) @ abs(B[:, 32 * e:32 * e + 32]).T)[0]
        assert (np.abs(host(c[e, r]) - want) <= 1e-5 * mag).all()


def test_weights_of_many_experts(gpu_lib):
    """Weights whose codes pass 2^32 bytes: the few-row products and the rows' products of the last experts."""
    need(20)
    E, n, k = 1024, 2112, 4096                             # 4.4 GB of codes
    b = codes((E, n, k), 2)
    assert b[0].numel() > 1 << 32
    ids = torch.tensor([[0, E - 1], [E - 2, 500]], dtype=torch.int32, device="cuda")
    offsets, slots, rows = gpu_lib.fp4_expert_sort(ids, E, 1)
    a = codes((4, k), 3)
    c = gpu_lib.fp4_gemm_experts(offsets, *a, *b)
    x = torch.randn((4, k), device="cuda").bfloat16()
    few = gpu_lib.fp4_matvec_experts(offsets, x, *b)
    for t in range(2):
        for j in range(2):
            e, r = int(ids[t, j]), int(rows[t, j])
            W = value(b[0][e], b[1][e])
            for got, v in ((c, value(a[0][r], a[1][r])), (few, host(x[r])[None].astype(np.float64))):
                assert (np.abs(host(got[r]) - (v @ W.T)[0]) <= 1e-5 * (abs(v) @ abs(W).T)[0]).all()
