"""GPU checks of the products' epilogue and its gradients against float64.

Bounds: the product 1e-5 sum |a b|; each fp32 addition half a step; the
activations' values and slopes in fp32 within 1e-6 |z| and 1e-5 (the hardware's
exponential, reciprocal and the fit of the normal tail are within 5e-7 together;
a slope multiplies that by at most 35, where 1 - s of the tanh form meets
x u'(x) at x = 5); one rounding to bf16."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import act as A
from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N

pytestmark = pytest.mark.gpu
H, U = 2.0 ** -8, 2.0 ** -24
ACTS = [A.NONE, A.RELU, A.GELU, A.GELU_TANH, A.SILU]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()


def operand(rows, k, seed):
    """Random codes whose decoded rows have a norm near sqrt(k) / 3, so that z spans the activations' bends."""
    rng = np.random.default_rng(seed)
    return rng.integers(0, 256, (rows, k // 2), dtype=np.uint8), rng.integers(122, 126, (rows, k // 32), dtype=np.uint8)


def expected(ref, e, k, act, bias, res):
    """(y, its bound in fp32, z, its bound)."""
    z, tol = ref, 1e-5 * e + k * 2.0 ** -150
    if bias is not None:
        z = z + bias
        tol = tol + U * (np.abs(z) + tol)
    y = A.value(z, act)
    tz = tol
    if act not in (A.NONE, A.RELU):
        tol = 1.2 * tol + 1e-6 * np.abs(z)                 # slopes are below 1.13
    if res is not None:
        y = y + res
        tol = tol + U * (np.abs(y) + tol)
    return y, tol, z, tz


def check(got, want, tol, f32):
    bound = tol + (0 if f32 else H * (np.abs(want) + tol))
    bad = ~(np.abs(host(got) - want) <= bound + 2.0 ** -140)
    assert not bad.any(), f"{bad.sum()} outside the bound, first {np.argwhere(bad)[0]}"


GEMMS = [(1, 32, 32), (5, 64, 64), (33, 96, 96), (100, 160, 224), (256, 256, 256), (257, 288, 288), (300, 544, 512), (64, 32, 1056),
         (513, 320, 1280), (31, 64, 0), (700, 96, 4096)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", GEMMS)
def test_gemm_act(gpu_lib, m, n, k, act):
    rng = np.random.default_rng(m + n)
    a, b = operand(m, k, 1), operand(n, k, 2)
    ref, e = G.gemm_ref(*a, *b)
    scale = 2.0 / max(float(np.sqrt((ref ** 2).mean())), 1.0)
    down = int(round(np.log2(scale)))                      # z of a few units: a power of two from b's scales
    b = (b[0], (b[1].astype(int) + down).astype(np.uint8))
    ref, e = G.gemm_ref(*a, *b)
    bias, res = rng.normal(size=n).astype(np.float32), rng.normal(size=(m, n)).astype(np.float32)
    rt = torch.zeros((m, n + 8), dtype=torch.bfloat16, device="cuda")[:, :n]
    rt.copy_(dev(res))
    ab = [*map(dev, a), *map(dev, b)]
    for bt, r, f32, z in ((None, None, True, False), (dev(bias), None, False, True), (dev(bias).bfloat16(), rt, True, True),
                          (None, rt, False, False), (dev(bias).bfloat16(), rt, False, True)):
        y = torch.full((m, n + 8), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        got, got_z = gpu_lib.fp4_gemm_act(*ab, act, bias=bt, residual=r, y=y[:, :n], emit_z=z)
        want, tol, wz, tz = expected(ref, e, k, act, None if bt is None else host(bt).astype(np.float64),
                                     None if r is None else host(r).astype(np.float64))
        check(got, want, tol, f32)
        assert (host(y)[:, n:] == 7).all() and (got_z is None) == (not z)
        if z:
            check(got_z, wz, tz, False)


GEMMS_LARGE = [(2081, 2080, 256, A.GELU), (1030, 4128, 288, A.SILU), (4100, 1056, 96, A.RELU), (2050, 2112, 0, A.GELU_TANH),
               (1100, 4096, 1056, A.NONE)]


@pytest.mark.parametrize("m,n,k,act", GEMMS_LARGE)
def test_gemm_act_of_many_tiles(gpu_lib, m, n, k, act):
    test_gemm_act(gpu_lib, m, n, k, act)


@pytest.mark.parametrize("k", [96, 288, 1024, 2080])
def test_rows_do_not_depend_on_the_tile_size(gpu_lib, k):
    """A product of few tiles and the same rows of one of many: the same sums in the same order."""
    a, b = [dev(v) for v in operand(2081, k, 1)], [dev(v) for v in operand(2080, k, 2)]
    y, z = gpu_lib.fp4_gemm_act(*a, *b, A.GELU, emit_z=True)
    for m, n in ((1, 2080), (70, 2080), (2081, 96)):
        got, got_z = gpu_lib.fp4_gemm_act(*[v[:m] for v in a], *[v[:n] for v in b], A.GELU, emit_z=True)
        assert torch.equal(got, y[:m, :n]) and torch.equal(got_z, z[:m, :n])


def test_gemm_act_without_an_epilogue_is_the_product(gpu_lib):
    for m, n, k in ((64, 96, 256), (288, 320, 1024)):
        ab = [*map(dev, operand(m, k, 1)), *map(dev, operand(n, k, 2))]
        assert torch.equal(gpu_lib.fp4_gemm_act(*ab, dtype=torch.float32)[0], gpu_lib.fp4_gemm(*ab))


def test_gemm_act_onto_the_residual(gpu_lib):
    ab = [*map(dev, operand(300, 288, 1)), *map(dev, operand(96, 288, 2))]
    res = torch.randn(300, 96, device="cuda").bfloat16()
    want, _ = gpu_lib.fp4_gemm_act(*ab, A.SILU, residual=res)
    got, _ = gpu_lib.fp4_gemm_act(*ab, A.SILU, residual=res, y=res)
    assert got is res and torch.equal(res, want)


FEW = [(1, 1, 32), (1, 16, 64), (3, 33, 128), (5, 64, 544), (16, 100, 1024), (17, 48, 2080), (33, 19, 1056), (48, 16, 512), (64, 130, 640),
       (1, 4096, 4096), (2, 515, 4128), (64, 32, 14336), (4, 20000, 256), (3, 40, 0)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", FEW)
def test_matvec_act(gpu_lib, m, n, k, act, kind):
    rng = np.random.default_rng(m + n)
    bits = synthetic.tensor((m, max(k, 32)), seed=k)[:, :k]
    if kind == "bf16":
        x64, x, scales = F.bf16_bits_to_f64(bits), dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16), None
    elif k == 0:
        return
    else:
        c, s = N.encode_e4m3(bits)
        x64, x, scales = N.decode_e4m3(c, s), dev(c), dev(s)
    w = operand(n, k, 2)
    down = int(round(np.log2(2.0 / max(np.sqrt(k), 1.0))))
    w = (w[0], (w[1].astype(int) + down).astype(np.uint8))
    W = F.decode(*w)
    ref, e = x64 @ W.T, abs(x64) @ abs(W).T
    bias, res = rng.normal(size=n).astype(np.float32), rng.normal(size=(m, n)).astype(np.float32)
    rt = torch.zeros((m, n + 5), dtype=torch.bfloat16, device="cuda")[:, :n]
    rt.copy_(dev(res))
    for bt, r, f32 in ((None, None, True), (dev(bias), rt, False), (dev(bias).bfloat16(), None, False), (None, rt, True)):
        y = torch.full((m, n + 3), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        got = gpu_lib.fp4_matvec_act(x, *map(dev, w), act, x_scales=scales, bias=bt, residual=r, y=y[:, :n])
        want, tol, _, _ = expected(ref, e, k, act, None if bt is None else host(bt).astype(np.float64),
                                   None if r is None else host(r).astype(np.float64))
        check(got, want, tol, f32)
        assert (host(y)[:, n:] == 7).all()


GRADS = [(1, 32), (2, 64), (7, 96), (8, 128), (33, 160), (64, 256), (65, 288), (300, 1056), (1000, 64), (4096, 32), (129, 4096),
         (515, 14336)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", GRADS)
def test_act_backward(gpu_lib, m, n, act, f32):
    rng = np.random.default_rng(m + n)
    z = torch.zeros((m, n + 8), dtype=torch.bfloat16, device="cuda")[:, :n]
    z.copy_(dev((2.5 * rng.normal(size=(m, n))).astype(np.float32)))
    dy = torch.zeros((m, n + 8), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")[:, :n]
    dy.copy_(dev(rng.normal(size=(m, n)).astype(np.float32)))
    dy64, slope = host(dy).astype(np.float64), A.slope(host(z), act)
    tol = np.abs(dy64) * (0 if act in (A.NONE, A.RELU) else 1e-5) + U * np.abs(dy64 * slope)
    want = dy64 * slope
    dz, dbias = gpu_lib.fp4_act_backward(dy, z, act)
    check(dz, want, tol, False)
    mag, off = np.abs(want).sum(0), tol.sum(0)
    assert (np.abs(host(dbias) - want.sum(0)) <= off + (m + 40) * U * mag + 2.0 ** -140).all()
    prev = torch.randn(n, device="cuda")
    acc = prev.clone()
    gpu_lib.fp4_act_backward(dy, z, act, accumulate=True, dbias=acc)
    assert (np.abs(host(acc) - host(prev) - want.sum(0)) <= off + (m + 41) * U * (mag + np.abs(host(prev)))).all()
    only, none = gpu_lib.fp4_act_backward(dy, z, act, emit_dbias=False)
    assert none is None and torch.equal(only, dz)
    again = gpu_lib.fp4_act_backward(dy, z, act)
    assert torch.equal(again[0], dz) and torch.equal(again[1], dbias)


@pytest.mark.parametrize("act", ACTS)
def test_slopes_over_every_bf16(gpu_lib, act):
    """Every finite bf16 z: the slope within its bound, 0 or 1 far out; NaN stays NaN."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    z = dev(bits.view(np.int16)).view(torch.bfloat16).reshape(2048, 32)
    dz, _ = gpu_lib.fp4_act_backward(torch.ones((2048, 32), device="cuda"), z, act, emit_dbias=False)
    zf, got = host(z), host(dz)
    fine = np.isfinite(zf)
    with np.errstate(over="ignore", invalid="ignore"):
        x = np.clip(np.where(fine, zf, 0).astype(np.float64), -1e3, 1e3)            # slopes are constant out there
    want = A.slope(x, act)
    tol = 0 if act in (A.NONE, A.RELU) else 1e-5
    assert (np.abs(got - want) <= tol + H * (np.abs(want) + tol))[fine].all()
    if act != A.NONE:
        assert np.isnan(got[np.isnan(zf)]).all()
        assert (got[zf == np.inf] == 1).all() and (got[zf == -np.inf] == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_values_over_every_bf16(gpu_lib, act):
    """act(z) of every finite bf16 z, put into z by the bias of an empty product."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    zf = F.bf16_bits_to_f64(bits)
    bias = dev(bits.view(np.int16)).view(torch.bfloat16)
    empty = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((1, 0), (1, 0), (65536, 0), (65536, 0))]
    got = host(gpu_lib.fp4_gemm_act(*empty, act, bias=bias, dtype=torch.float32)[0])[0]
    fine = np.isfinite(zf)
    x = np.where(fine, zf, 0)
    with np.errstate(over="ignore"):
        want = x if act == A.NONE else np.where(np.abs(x) > 1e3, np.maximum(x, 0), A.value(np.clip(x, -1e3, 1e3), act))
    tol = 0 if act in (A.NONE, A.RELU) else 1e-6
    assert (np.abs(got - want) <= tol * np.abs(np.where(x < -1e3, 0, x)) + 2.0 ** -140)[fine].all()
    assert np.isnan(got[np.isnan(zf)]).all() and got[zf == np.inf] == np.inf
    assert got[zf == -np.inf] == (-np.inf if act == A.NONE else 0)


def test_no_rows(gpu_lib):
    z = torch.zeros((0, 64), device="cuda").bfloat16()
    dbias = torch.ones(64, device="cuda")
    gpu_lib.fp4_act_backward(z, z, A.GELU, accumulate=True, dbias=dbias)
    assert (host(dbias) == 1).all()
    dz, dbias = gpu_lib.fp4_act_backward(z, z, A.GELU, dbias=dbias)
    assert dz.shape == (0, 64) and (host(dbias) == 0).all()
    codes = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((0, 32), (0, 2), (64, 32), (64, 2))]
    assert gpu_lib.fp4_gemm_act(*codes, A.GELU)[0].shape == (0, 64)
