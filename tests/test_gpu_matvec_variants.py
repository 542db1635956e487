"""Every variant of the few-row products' kernel against float64: widths of
several rounds of tiles, x that does not fit LDS beside the partial sums (each
wave then brings its own steps of it), one to four tiles of rows of x, one and
two tiles of W a wave, items of one, two and four steps, reductions that end
inside a step, scales off a word boundary.

The bounds are those of the GEMM, 1e-5 sum |a b| (every decoded value is exact
in bf16, the sums are fp32), carried through the roundings of the gated form.
Each call is made twice: the sums have a fixed order, so the bytes are the same.
"""

import numpy as np
import pytest
import torch

import synthetic
from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N
from oracle import nvfp4 as NV

pytestmark = pytest.mark.gpu
H = 2.0 ** -8                                            # half a bf16 step

# rows of x, rows of W (gated: of W1), length, bytes that the scales are off a word boundary
SHAPES = [
    # x staged in LDS: items of four, two and one steps, partial steps, odd scale addresses, several meetings
    (3, 9001, 1536, 0), (3, 18002, 1536, 0), (5, 8201, 512, 0), (1, 700, 1024, 0), (16, 4100, 4096, 0), (2, 900, 768, 0),
    (4, 9000, 256, 0), (3, 130, 384, 0), (6, 8197, 640, 0), (7, 5000, 288, 0), (12, 77, 992, 0), (9, 8200, 1024, 1),
    (1, 14336, 1024, 0), (5, 40001, 256, 0), (16, 14336, 1024, 0), (1, 33000, 96, 0),
    # sixteen rows and fewer, brought by each wave
    (16, 8209, 4608, 0), (16, 4103, 4608, 0), (9, 4200, 8192, 0), (16, 70, 4608, 0), (16, 50, 4640, 0), (13, 40, 6144, 2),
    # two, three and four tiles of rows
    (17, 8217, 1536, 0), (32, 4105, 2048, 0), (25, 60, 640, 0), (30, 4100, 416, 0), (20, 33000, 384, 0),
    (33, 8203, 1152, 0), (48, 4108, 512, 0), (40, 90, 896, 0), (35, 4099, 288, 0), (40, 17000, 256, 0), (33, 260, 4096, 0),
    (49, 8220, 1024, 0), (64, 4101, 640, 0), (55, 33, 768, 0), (64, 4200, 160, 0), (50, 300, 512, 3), (64, 16400, 384, 0),
]
KINDS = ["bf16", "e4m3"]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def off_by(a, by):
    """The tensor `a` at an address `by` bytes past a word boundary."""
    flat = torch.cat([torch.zeros(by, dtype=torch.uint8, device="cuda"), a.flatten()])
    return flat[by:].view(a.shape)


def activations(m, k, seed, kind):
    """(float64 values, x, x_scales), all on the device."""
    b = synthetic.tensor((m, k), seed=seed, outlier_rate=0.002, outlier_scale=20.0)
    if kind == "bf16":
        return dev(F.bf16_bits_to_f64(b)), dev(b.view(np.int16)).view(torch.bfloat16), None
    codes, scales = N.encode_e4m3(b)
    return dev(N.decode_e4m3(codes, scales)), dev(codes), dev(scales)


def random_codes(n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return g, torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)


def values(codes, scales, group):
    """float64 values of packed E2M1 codes under one float64 scale a group."""
    pairs = dev(F.decode_nibble(F.unpack_nibbles(np.arange(256, dtype=np.uint8)[:, None])))   # of every byte
    n, half = codes.shape
    v = pairs[codes.int()].view(n, 2 * half // group, group)
    return (v * scales[..., None]).view(n, 2 * half)


def e8m0(b):
    return torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), b.int() - 127)


def e4m3(b):
    return dev(NV.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64))[b.int()]


def check(got, x64, w64, prev=None):
    ref, e = x64 @ w64.t(), x64.abs() @ w64.abs().t()
    ok = G.within_bound(host(got), host(ref), host(e), c_prev=prev, k=x64.shape[1])
    assert ok.all(), f"{(~ok).sum()} outside the bound, first {np.argwhere(~ok)[0]}"


@pytest.mark.parametrize("m,n,k,off", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_matvec(gpu_lib, m, n, k, off, kind):
    x64, x, xs = activations(m, k, 31, kind)
    g, codes = random_codes(n, k, 32)
    scales = torch.randint(116, 124, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    w64, at = values(codes, e8m0(scales), 32), off_by(scales, off)
    c = gpu_lib.fp4_matvec(x, codes, at, xs)
    check(c, x64, w64)
    assert torch.equal(gpu_lib.fp4_matvec(x, codes, at, xs), c)
    prev = host(c).copy()
    check(gpu_lib.fp4_matvec(x, codes, at, xs, c=c, accumulate=True), x64, w64, prev)


@pytest.mark.parametrize("m,n,k,off", SHAPES)
def test_nv_matvec(gpu_lib, m, n, k, off):
    x64, x, _ = activations(m, k, 33, "bf16")
    g, codes = random_codes(n, k, 34)
    scales = torch.randint(0, 0x7F, (n, k // 16), dtype=torch.uint8, device="cuda", generator=g)
    factors = torch.exp2(-12 + 4 * torch.rand((n + 255) // 256, device="cuda", generator=g))
    w64 = values(codes, e4m3(scales), 16) * factors.double().repeat_interleave(256)[:n, None]
    at = off_by(scales, off)
    c = gpu_lib.fp4_nv_matvec(x, codes, at, factors)
    check(c, x64, w64)
    assert torch.equal(gpu_lib.fp4_nv_matvec(x, codes, at, factors), c)
    prev = host(c).copy()
    check(gpu_lib.fp4_nv_matvec(x, codes, at, factors, c=c, accumulate=True), x64, w64, prev)


@pytest.mark.parametrize("m,f,d,off", SHAPES)
@pytest.mark.parametrize("kind", KINDS)
def test_swiglu_matvec(gpu_lib, m, f, d, off, kind):
    x64, x, xs = activations(m, d, 35, kind)
    g, codes = random_codes(2 * f, d, 36)
    top = 121 - int(np.log2(d) / 2)                       # a and b of order one
    scales = torch.randint(top - 2, top + 2, (2 * f, d // 32), dtype=torch.uint8, device="cuda", generator=g)
    w64, at = values(codes, e8m0(scales), 32), off_by(scales, off)
    h = gpu_lib.fp4_swiglu_matvec(x, codes, at, xs)
    assert torch.equal(gpu_lib.fp4_swiglu_matvec(x, codes, at, xs), h)
    (a, b), (ea, eb) = (x64 @ w64.t()).split(f, 1), (x64.abs() @ w64.abs().t()).split(f, 1)
    silu = a * torch.sigmoid(a)
    # a and b off by the sum's bound and a bf16 rounding; |SiLU'| <= 1.1; the gate's own fp32
    # roundings (below 8 of 2^-24) and h's bf16 rounding
    da, db = H * a.abs() + 1e-5 * ea, H * b.abs() + 1e-5 * eb
    away = 1.1 * da * (b.abs() + db) + silu.abs() * db
    assert ((h.double() - silu * b).abs() <= away + (H + 2.0 ** -20) * ((silu * b).abs() + away) + 2.0 ** -133).all()
