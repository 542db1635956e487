"""GPU checks of the few-row products against float64: fp4_matvec and
fp4_nv_matvec within the GEMM bound 1e-5 sum |a b| (every decoded value is
exact in bf16, the sums are fp32), fp4_swiglu_matvec within that bound carried
through the two bf16 roundings and the gate."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N
from oracle import nvfp4 as NV
from oracle import quant as Q
from oracle import swiglu as S
import synthetic

pytestmark = pytest.mark.gpu
H = 2.0 ** -8                                            # half a bf16 step


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dev16(b):
    return dev(b.view(np.int16)).view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def weights(n, k, seed, wide=False):
    """Random codes (every nibble) and scale bytes; `wide`: over most of the range."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    lo, hi = (60, 190) if wide else (116, 124)
    return codes, rng.integers(lo, hi, (n, k // 32), dtype=np.uint8)


def activations(m, k, seed, kind):
    """(float64 values, x, x_scales) on the device."""
    b = synthetic.tensor((m, k), seed=seed, outlier_rate=0.002, outlier_scale=20.0)
    if kind == "bf16":
        return F.bf16_bits_to_f64(b), dev16(b), None
    codes, scales = N.encode_e4m3(b)
    return N.decode_e4m3(codes, scales), dev(codes), dev(scales)


def check(got, x, w, prev=None):
    ref, e = x @ w.T, np.abs(x) @ np.abs(w).T
    ok = G.within_bound(host(got), ref, e, c_prev=prev, k=x.shape[1])
    assert ok.all(), f"{(~ok).sum()} outside the bound, first {np.argwhere(~ok)[0]}"


SHAPES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (1, 5, 160), (3, 33, 128), (5, 64, 544), (16, 100, 1024), (17, 48, 2080),
          (31, 31, 256), (32, 257, 4096), (33, 19, 1056), (48, 16, 512), (64, 130, 640), (1, 1000, 8192), (64, 32, 14336),
          (7, 4096, 288), (2, 515, 4128), (1, 9000, 512), (4, 20000, 256), (16, 8200, 4096), (3, 12289, 1536), (9, 6000, 6144),
          (50, 5000, 1280), (20, 4200, 384), (16, 40, 4544), (16, 40, 4576), (12, 8300, 8192), (33, 8192, 256),
          (64, 8209, 128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_matvec(gpu_lib, m, n, k, kind):
    x64, x, xs = activations(m, k, 1, kind)
    codes, scales = weights(n, k, 2)
    w64 = F.decode(codes, scales)
    c = gpu_lib.fp4_matvec(x, dev(codes), dev(scales), xs)
    check(c, x64, w64)
    prev = host(c).copy()
    out = gpu_lib.fp4_matvec(x, dev(codes), dev(scales), xs, c=c, accumulate=True)
    assert out is c
    check(c, x64, w64, prev=prev)


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("panels", [False, True])
def test_nv_matvec(gpu_lib, m, n, k, panels):
    x64, x, _ = activations(m, k, 3, "bf16")
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    scales = rng.integers(0, 0x7F, (n, k // 16), dtype=np.uint8)       # every E4M3 scale, subnormals and zero too
    fac = (2.0 ** rng.uniform(-12, -8, (n + 255) // 256 if panels else 1)).astype(np.float32)
    c = gpu_lib.fp4_nv_matvec(x, dev(codes), dev(scales), dev(fac))
    w64 = NV.decode(codes, scales) * np.repeat(fac.astype(np.float64), 256 if fac.size > 1 else n)[:n, None]
    check(c, x64, w64)
    prev = host(c).copy()
    gpu_lib.fp4_nv_matvec(x, dev(codes), dev(scales), dev(fac), c=c, accumulate=True)
    check(c, x64, w64, prev=prev)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_matvec_wide_scales(gpu_lib, kind):
    """Scale bytes over most of the E8M0 range (bf16 holds every value exactly)."""
    x64, x, xs = activations(3, 320, 5, kind)
    codes, scales = weights(70, 320, 6, wide=True)
    check(gpu_lib.fp4_matvec(x, dev(codes), dev(scales), xs), x64, F.decode(codes, scales))
    # the lowest scales: weights down to 2^-128, products in the fp32 subnormal range
    scales[:] = np.arange(scales.size, dtype=np.uint8).reshape(scales.shape) % 6
    check(gpu_lib.fp4_matvec(x, dev(codes), dev(scales), xs), x64, F.decode(codes, scales))


def test_matvec_every_code_and_scale(gpu_lib):
    """x = unit rows pick single weights: each nibble under each scale byte up to
    2^126 (6 of them stay below 2^128 through byte 252), exactly."""
    k = 64
    codes = np.tile(np.arange(16, dtype=np.uint8)[:, None] * 17, (1, k // 2))
    codes = np.concatenate([codes] * 2)[:16]
    x = np.zeros((2, k), np.float32)
    x[0, 5] = x[1, 40] = 1.0
    xd = dev16(synthetic.bf16_bits(x))
    for byte in range(0, 253):
        scales = np.full((16, 2), byte, np.uint8)
        got = host(gpu_lib.fp4_matvec(xd, dev(codes), dev(scales))).astype(np.float64)
        want = (x.astype(np.float64) @ F.decode(codes, scales).T)
        assert np.array_equal(got, want), byte


@pytest.mark.parametrize("m,n,k", [(4, 20, 96), (20, 20, 96), (40, 20, 256), (60, 8200, 128), (16, 20, 4640)])
def test_non_finite_rows_stay_apart(gpu_lib, m, n, k):
    """An infinity or NaN in one row of x does not reach the other rows, nor do
    values in the row's padding."""
    codes, scales = weights(n, k, 7)
    xb = synthetic.tensor((m, k + 32), seed=8)
    xd = dev16(xb).clone()
    xd[1, 3] = float("inf")
    xd[2, k - 6] = float("nan")
    xd[:, k:] = float("nan")
    got = host(gpu_lib.fp4_matvec(xd[:, :k], dev(codes), dev(scales)))
    x64 = F.bf16_bits_to_f64(xb)[:, :k]
    ref, e = x64 @ F.decode(codes, scales).T, np.abs(x64) @ np.abs(F.decode(codes, scales)).T
    rest = [0, *range(3, m)]
    assert G.within_bound(got[rest], ref[rest], e[rest], k=k).all()
    assert np.isnan(got[2]).all() and not np.isfinite(got[1]).any()


def test_strided_operands_leave_padding(gpu_lib):
    m, n, k = 5, 37, 160
    codes, scales = weights(n, k, 9)
    xb = synthetic.tensor((m, 200), seed=10)
    buf = torch.full((m + 1, n + 6), -3.0, device="cuda")
    c = buf[:m, 2:2 + n]
    gpu_lib.fp4_matvec(dev16(xb)[:, 8:8 + k], dev(codes), dev(scales), c=c)
    check(c, F.bf16_bits_to_f64(xb)[:, 8:8 + k], F.decode(codes, scales))
    o = host(buf)
    assert (o[m] == -3).all() and (o[:, :2] == -3).all() and (o[:, 2 + n:] == -3).all()


@pytest.mark.parametrize("m,k", [(1, 512), (3, 1024), (5, 160), (20, 512), (40, 256)])
@pytest.mark.parametrize("by", [1, 2, 4])
def test_scales_at_any_address(gpu_lib, m, k, by):
    """Scale rows that start off a word boundary (a slice of a larger buffer)."""
    mx, n = gpu_lib, 50
    x64, x, _ = activations(m, k, 20, "bf16")
    codes, scales = weights(n, k, 21)
    at = lambda a: torch.cat([torch.zeros(by, dtype=torch.uint8, device="cuda"), dev(a).flatten()])[by:].view(a.shape)  # noqa: E731
    check(mx.fp4_matvec(x, dev(codes), at(scales)), x64, F.decode(codes, scales))
    s4 = np.random.default_rng(22).integers(0, 0x7F, (n, k // 16), dtype=np.uint8)
    check(mx.fp4_nv_matvec(x, dev(codes), at(s4), torch.ones(1, device="cuda")), x64, NV.decode(codes, s4))
    xe, xc, xs = activations(m, k, 23, "e4m3")
    check(mx.fp4_matvec(xc, dev(codes), at(scales), at(host(xs))), xe, F.decode(codes, scales))


def test_empty_reduction_and_empty_outputs(gpu_lib):
    mx = gpu_lib
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = torch.empty((3, 0), dtype=torch.bfloat16, device="cuda")
    c = torch.full((3, 7), 2.0, device="cuda")
    mx.fp4_matvec(x, u8(7, 0), u8(7, 0), c=c, accumulate=True)
    assert (host(c) == 2).all()
    mx.fp4_matvec(x, u8(7, 0), u8(7, 0), c=c)
    assert (host(c) == 0).all()
    h = torch.full((3, 2), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.fp4_swiglu_matvec(x, u8(4, 0), u8(4, 0), h=h)
    assert (host(h.float()) == 0).all()
    y = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert mx.fp4_matvec(y, u8(5, 32), u8(5, 2)).shape == (0, 5)
    assert mx.fp4_matvec(torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda"), u8(0, 32), u8(0, 2)).shape == (2, 0)


@pytest.mark.parametrize("m,f,d", [(1, 1, 32), (1, 16, 64), (2, 33, 160), (5, 100, 1056), (16, 48, 4096), (17, 31, 288),
                                   (40, 65, 512), (64, 256, 2048), (1, 1792, 4096)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_swiglu_matvec(gpu_lib, m, f, d, kind):
    x64, x, xs = activations(m, d, 11, kind)
    rng = np.random.default_rng(12)
    codes = rng.integers(0, 256, (2 * f, d // 2), dtype=np.uint8)
    top = 121 - int(np.log2(d) / 2)                       # a and b of order one
    scales = rng.integers(top - 2, top + 2, (2 * f, d // 32), dtype=np.uint8)
    w = F.decode(codes, scales)
    h = host(gpu_lib.fp4_swiglu_matvec(x, dev(codes), dev(scales), xs).float()).astype(np.float64)
    ab, e = x64 @ w.T, np.abs(x64) @ np.abs(w).T
    a, b, ea, eb = ab[:, :f], ab[:, f:], e[:, :f], e[:, f:]
    sig = 1 / (1 + np.exp(-a))
    silu = a * sig
    # a and b off by the sum's bound and a bf16 rounding; |SiLU'| <= 1.1; the gate's own fp32
    # roundings (below 8 of 2^-24) and h's bf16 rounding
    da, db = H * np.abs(a) + 1e-5 * ea, H * np.abs(b) + 1e-5 * eb
    off = 1.1 * da * (np.abs(b) + db) + np.abs(silu) * db
    assert (np.abs(h - silu * b) <= off + (H + 2.0 ** -20) * (np.abs(silu * b) + off) + 2.0 ** -133).all()


def test_swiglu_matvec_is_the_gate_of_the_products(gpu_lib):
    """h from fp4_matvec's a and b through the oracle's gate: the same bits
    wherever neither bf16 rounding of a sum is near a tie."""
    m, f, d = 9, 70, 544
    x64, x, _ = activations(m, d, 13, "bf16")
    codes, scales = weights(2 * f, d, 14)
    scales = (scales - 5).astype(np.uint8)
    ab = x64 @ F.decode(codes, scales).T
    e = np.abs(x64) @ np.abs(F.decode(codes, scales)).T
    bits = lambda v: S.f32_to_bf16_rne(v.astype(np.float32))  # noqa: E731
    sure = bits(ab - 1e-5 * e) == bits(ab + 1e-5 * e)
    h = gpu_lib.fp4_swiglu_matvec(x, dev(codes), dev(scales))
    got = host(h.view(torch.int16)).view(np.uint16)
    want = S.swiglu_h(bits(ab[:, :f]), bits(ab[:, f:]))
    ok = sure[:, :f] & sure[:, f:]
    assert ok.mean() > 0.5
    assert np.array_equal(got[ok], want[ok])


def test_matvec_agrees_with_the_gemm(gpu_lib):
    """The decoded MXFP4 rows as bf16 x: fp4_gemm on the codes and fp4_matvec on
    the values are the same contraction."""
    mx = gpu_lib
    xb = synthetic.tensor((32, 512), seed=15)
    wb = synthetic.tensor((96, 512), std=0.02, seed=16)
    xc, xsc = Q.quantize_rows(xb)
    wq = mx.fp4_quantize_w2d32(dev16(wb))
    x64 = F.decode(xc, xsc)
    x = dev16(synthetic.bf16_bits(x64.astype(np.float32)))    # exact
    w64 = F.decode(host(wq[0]), host(wq[1]))
    check(mx.fp4_matvec(x, wq[0], wq[1]), x64, w64)
    check(mx.fp4_gemm(dev(xc), dev(xsc), wq[0], wq[1]), x64, w64)
    nv = mx.fp4_nv_quantize_w2d16(dev16(wb))
    check(mx.fp4_nv_matvec(x, nv[0], nv[1], nv[4]), x64, NV.decode(host(nv[0]), host(nv[1])) * float(host(nv[4])[0]))


def test_weights_past_32_bit_offsets(gpu_lib):
    """n * k / 2 above 2^32 bytes: sampled rows on both sides of the border."""
    n, k = 540_673, 16384
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(116, 124, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    x64, x, _ = activations(2, k, 17, "bf16")
    c = gpu_lib.fp4_matvec(x, codes, scales)
    rows = torch.tensor([0, 15, 262143, 524287, 524288, 524289, 540656, 540671, 540672], device="cuda")
    w64 = F.decode(host(codes[rows]), host(scales[rows]))
    check(c[:, rows], x64, w64)
    del codes, scales, c
    torch.cuda.empty_cache()


def test_refusals_of_the_binding(gpu_lib):
    mx = gpu_lib
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    w, sc = u8(6, 32), u8(6, 2)
    f1 = torch.ones(1, device="cuda")
    bad = [
        lambda: mx.fp4_matvec(x.cpu(), w, sc), lambda: mx.fp4_matvec(x.float(), w, sc), lambda: mx.fp4_matvec(x[:, :32], w, sc),
        lambda: mx.fp4_matvec(x, w, sc[:5]), lambda: mx.fp4_matvec(x, w.int(), sc), lambda: mx.fp4_matvec(x, w.t(), sc),
        lambda: mx.fp4_matvec(x, w, sc, x_scales=u8(2, 2)), lambda: mx.fp4_matvec(u8(2, 64), w, sc, x_scales=u8(2, 1)),
        lambda: mx.fp4_matvec(u8(2, 64), w, sc), lambda: mx.fp4_matvec(x, w, sc, accumulate=True),
        lambda: mx.fp4_matvec(x, w, sc, c=torch.zeros((2, 5), device="cuda")),
        lambda: mx.fp4_matvec(x, w, sc, c=torch.zeros((2, 6), device="cuda").bfloat16()),
        lambda: mx.fp4_matvec(torch.zeros((65, 64), dtype=torch.bfloat16, device="cuda"), w, sc),
        lambda: mx.fp4_nv_matvec(x, w, u8(6, 2), f1), lambda: mx.fp4_nv_matvec(x, w, u8(6, 4), f1.double()),
        lambda: mx.fp4_nv_matvec(x, w, u8(6, 4), torch.ones(3, device="cuda")),
        lambda: mx.fp4_swiglu_matvec(x, u8(5, 32), u8(5, 2)),
        lambda: mx.fp4_swiglu_matvec(x, w, sc, h=torch.zeros((2, 4), dtype=torch.bfloat16, device="cuda")),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(mx.Fp4Error):
            f()
            pytest.fail(f"call {k} was not refused")


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(gpu_lib, seed):
    """Shapes drawn over the whole range (logarithmic), each call once."""
    mx, rng = gpu_lib, np.random.default_rng(1000 + seed)
    log = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))  # noqa: E731
    m, n, k = log(1, 64), log(1, 3000), 32 * log(1, 300)
    kind = ("bf16", "e4m3")[seed % 2]
    x64, x, xs = activations(m, k, 2000 + seed, kind)
    codes, scales = weights(n, k, 3000 + seed)
    check(mx.fp4_matvec(x, dev(codes), dev(scales), xs), x64, F.decode(codes, scales))
    if kind == "bf16":
        s4 = rng.integers(0, 0x7F, (n, k // 16), dtype=np.uint8)
        check(mx.fp4_nv_matvec(x, dev(codes), dev(s4), torch.ones(1, device="cuda")), x64, NV.decode(codes, s4))
    if n % 2 == 0:
        # the gate, in the 2-norm: two rounded factors and the result
        lo = (scales - 4 - int(np.log2(k) / 2)).astype(np.uint8)
        ab = x64 @ F.decode(codes, lo).T
        a, b = ab[:, :n // 2], ab[:, n // 2:]
        h = host(mx.fp4_swiglu_matvec(x, dev(codes), dev(lo), xs).float()).astype(np.float64)
        want = a / (1 + np.exp(-a)) * b
        assert np.linalg.norm(h - want) <= 3 * H * np.linalg.norm(want) + 1e-30
