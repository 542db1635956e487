"""GPU checks of the experts' products against float64 within the GEMM bound 1e-5
sum |a b|, and of the gated producer byte for byte against the plain one expert
by expert."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import act as A
from oracle import experts as X
from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N
from oracle import quant as Q
from test_gpu_matvec_variants import KINDS, SHAPES

pytestmark = pytest.mark.gpu
H = 2.0 ** -8                                            # half a bf16 step


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()


def codes(shape, seed):
    """Random codes (every nibble) and scale bytes of [..., k] values."""
    rng = np.random.default_rng(seed)
    *lead, k = shape
    return rng.integers(0, 256, (*lead, k // 2), dtype=np.uint8), rng.integers(116, 126, (*lead, k // 32), dtype=np.uint8)


def segments(sizes, align, rows=None):
    """(offsets, rows of the buffers) of experts with so many tokens."""
    padded = [-(-s // align) * align for s in sizes]
    offsets = np.concatenate(([0], np.cumsum(padded))).astype(np.int32)
    return offsets, int(offsets[-1]) if rows is None else rows


def check(got, ref, e, k, f32=True):
    got = host(got)
    if f32:
        ok = G.within_bound(got, ref, e, k=k)
    else:                                                # the fp32 value rounded once
        tol = 1e-5 * e + k * 2.0 ** -150
        ok = np.abs(got - ref) <= tol + H * (np.abs(ref) + tol)
    assert ok.all(), f"{(~ok).sum()} outside the bound, first {np.argwhere(~ok)[0]}"


ROWS = [((1,), 32, 32), ((0, 3), 64, 64), ((5, 0, 1, 40), 32, 96), ((64, 32, 0, 0, 300), 96, 160), ((256, 257, 255), 256, 224),
        ((33, 1), 288, 256), ((100, 200, 300), 512, 288), ((7,) * 70, 64, 512), ((0,) * 65 + (9,), 320, 1056),
        ((513, 0, 700), 544, 768), ((3, 2000), 256, 4096), ((0, 0, 0), 64, 64)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("align,extra", [(1, 0), (1, 5), (32, 0), (32, 301)])
@pytest.mark.parametrize("sizes,n,k", ROWS)
def test_rows(gpu_lib, sizes, n, k, align, extra, f32):
    offsets, rows = segments(sizes, align)
    rows += extra
    a, b = codes((rows, k), 1), codes((len(sizes), n, k), 2)
    a2, b2 = codes((rows, k), 3), codes((len(sizes), n, k), 4)
    dtype = torch.float32 if f32 else torch.bfloat16
    ref, e = np.zeros((2, rows, n))
    ref2, e2 = np.zeros((2, rows, n))
    for i in range(len(sizes)):
        at = slice(offsets[i], offsets[i + 1])
        ref[at], e[at] = G.gemm_ref(a[0][at], a[1][at], b[0][i], b[1][i])
        ref2[at], e2[at] = G.gemm_ref(a2[0][at], a2[1][at], b2[0][i], b2[1][i])
    args = [dev(offsets), *map(dev, a), *map(dev, b)]
    c = torch.full((rows, n + 8), 7.0, dtype=dtype, device="cuda")
    out = gpu_lib.fp4_gemm_experts(*args, c=c[:, :n])
    check(out, ref, e, k, f32)
    assert (host(c)[:, n:] == 7).all() and (host(c)[offsets[-1]:, :n] == 0).all()
    check(gpu_lib.fp4_gemm_experts(*args, dtype=dtype, pair=[*map(dev, a2), *map(dev, b2)]), ref + ref2, e + e2, 2 * k, f32)


ROWS_LARGE = [((5000, 700, 0, 1281), 928, 96, 1, 0, True), ((5000, 700, 0, 1281), 928, 256, 1, 7, False),
              ((0, 3000, 257, 1, 900), 1440, 288, 32, 0, False), ((300,) * 20, 1056, 512, 32, 96, True)]


@pytest.mark.parametrize("sizes,n,k,align,extra,f32", ROWS_LARGE)
def test_rows_of_many_tiles(gpu_lib, sizes, n, k, align, extra, f32):
    test_rows(gpu_lib, sizes, n, k, align, extra, f32)


@pytest.mark.parametrize("k", [288, 1024])
def test_rows_do_not_depend_on_the_tile_size(gpu_lib, k):
    """An expert's rows beside those of others, in large tiles, and alone, in small ones."""
    offsets, rows = segments((5000, 0, 200, 1281), 1)
    a, b = [dev(v) for v in codes((rows, k), 1)], [dev(v) for v in codes((4, 928, k), 2)]
    pair = [dev(v) for v in (*codes((rows, k), 3), *codes((4, 928, k), 4))]
    both, one = gpu_lib.fp4_gemm_experts(dev(offsets), *a, *b, pair=pair), gpu_lib.fp4_gemm_experts(dev(offsets), *a, *b)
    at, alone = slice(offsets[2], offsets[3]), dev(np.array([0, 200], np.int32))
    few = [[v[at] for v in a], [v[2:3] for v in b], [v[at] for v in pair[:2]] + [v[2:3] for v in pair[2:]]]
    few = [[v.clone() for v in x] for x in few]            # slices may start off 16 bytes
    assert torch.equal(gpu_lib.fp4_gemm_experts(alone, *few[0], *few[1]), one[at])
    assert torch.equal(gpu_lib.fp4_gemm_experts(alone, *few[0], *few[1], pair=few[2]), both[at])


@pytest.mark.parametrize("sizes,n,k", [((64, 32, 96), 96, 256), ((300, 20), 288, 1024), ((33,), 256, 288)])
def test_rows_are_those_of_the_plain_product(gpu_lib, sizes, n, k):
    """One expert's rows by fp4_gemm: the same sums in the same order where K is whole steps, the same bound elsewhere."""
    offsets, rows = segments(sizes, 32)
    a, b = codes((rows, k), 1), codes((len(sizes), n, k), 2)
    got = gpu_lib.fp4_gemm_experts(dev(offsets), *map(dev, a), *map(dev, b))
    for i in range(len(sizes)):
        at = slice(offsets[i], offsets[i + 1])
        want = gpu_lib.fp4_gemm(dev(a[0][at]), dev(a[1][at]), dev(b[0][i]), dev(b[1][i]))
        if k % 256 == 0:
            assert torch.equal(got[at], want)
        else:
            _, e = G.gemm_ref(a[0][at], a[1][at], b[0][i], b[1][i])
            assert (np.abs(host(got[at]) - host(want)) <= 2e-5 * e).all()


def test_segments_that_are_not_ascending_stay_inside(gpu_lib):
    """Nothing is promised of their values, but that no other memory is touched:
    the columns beside C and the rows behind it keep what they hold."""
    a, b = codes((64, 64), 1), codes((4, 32, 64), 2)
    x = torch.randn(64, 64, device="cuda").bfloat16()
    for bad in ([0, 40, 20, 70, 90], [-5, 10, 1000, 20, 64], [2 ** 31 - 1] * 5, [-2 ** 31] * 5, [64, 0, 0, 0, 0]):
        offsets = dev(np.array(bad, np.int32))
        c = torch.full((80, 40), 7.0, device="cuda")
        gpu_lib.fp4_gemm_experts(offsets, *map(dev, a), *map(dev, b), c=c[:64, :32])
        assert (c[64:] == 7).all() and (c[:, 32:] == 7).all()
        c = torch.full((80, 40), 7.0, device="cuda")
        gpu_lib.fp4_matvec_experts(offsets, x, *map(dev, b), c=c[:64, :32])
        assert (c[64:] == 7).all() and (c[:, 32:] == 7).all()


WGRAD = [((1,), 32, 32), ((0, 5, 0, 64), 64, 96), ((256, 300, 31, 0, 700), 96, 288), ((33,) * 9, 288, 64), ((2000, 1), 256, 256),
         ((7, 8, 9, 250), 544, 320), ((0,) * 66 + (40,), 32, 64), ((0, 0), 64, 32),
         ((300, 40), 1312, 288), ((33, 0, 64), 96, 1312)]


@pytest.mark.parametrize("align,extra", [(32, 0), (32, 256), (256, 0)])
@pytest.mark.parametrize("sizes,m,n", WGRAD)
def test_wgrad(gpu_lib, sizes, m, n, align, extra):
    offsets, rows = segments(sizes, align)
    tokens = -(-rows // 256) * 256 + extra
    a, b = codes((m, tokens), 1), codes((n, tokens), 2)
    A, B = F.decode(*a), F.decode(*b)
    ref, e = np.zeros((2, len(sizes), m, n))
    for i in range(len(sizes)):
        at = slice(offsets[i], offsets[i + 1])
        ref[i], e[i] = A[:, at] @ B[:, at].T, abs(A[:, at]) @ abs(B[:, at]).T
    args = [dev(offsets), *map(dev, a), *map(dev, b)]
    check(gpu_lib.fp4_gemm_experts_wgrad(*args), ref, e, tokens)
    check(gpu_lib.fp4_gemm_experts_wgrad(*args, dtype=torch.bfloat16), ref, e, tokens, f32=False)
    prev = np.random.default_rng(5).normal(size=ref.shape).astype(np.float32)
    c = dev(prev)
    assert gpu_lib.fp4_gemm_experts_wgrad(*args, c=c, accumulate=True) is c
    assert G.within_bound(host(c), ref, e, c_prev=prev).all()
    assert all(np.array_equal(host(c)[i], prev[i]) for i in range(len(sizes)) if sizes[i] == 0)


WGRAD_LARGE = [((2000, 1, 0, 700), 1056, 1056, 32, 0), ((33,) * 9, 672, 704, 32, 256)]


@pytest.mark.parametrize("sizes,m,n,align,extra", WGRAD_LARGE)
def test_wgrad_of_many_tiles(gpu_lib, sizes, m, n, align, extra):
    test_wgrad(gpu_lib, sizes, m, n, align, extra)


def test_wgrad_does_not_depend_on_the_tile_size(gpu_lib):
    offsets, rows = segments((2000, 1, 0, 700, 40), 32)
    rows = -(-rows // 256) * 256
    a, b = [dev(v) for v in codes((1056, rows), 1)], [dev(v) for v in codes((1024, rows), 2)]
    want = gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), *a, *b)
    got = gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), *[v[:96] for v in a], *[v[:160] for v in b])
    assert torch.equal(got, want[:, :96, :160])


SWIGLU = [((32,), 32, 32), ((5, 0, 70, 300), 64, 96), ((256, 257), 96, 256), ((33, 1, 0), 160, 288), ((40,) * 67, 32, 64),
          ((600, 8), 288, 512), ((0, 0), 64, 64)]


@pytest.mark.parametrize("extra", [0, 32, 320])
@pytest.mark.parametrize("sizes,f,d", SWIGLU)
def test_swiglu_producer(gpu_lib, sizes, f, d, extra):
    """Each expert's rows byte for byte as fp4_swiglu_producer gives them; zeros behind."""
    offsets, rows = segments(sizes, 32)
    rows += extra
    if rows == 0:
        return
    xq, mask = codes((rows, d), 1), gpu_lib.fp4_sign_mask_from_seed(3)
    w = [Q.quantize_w2d32(synthetic.tensor((2 * f, d), std=0.05, seed=10 + i), 0.87)[:2] for i in range(len(sizes))]
    wc, ws = np.stack([c for c, _ in w]), np.stack([s for _, s in w])
    out = [torch.full(s, 9, dtype=t, device="cuda") for s, t in (((rows, f), torch.bfloat16), ((rows, f), torch.bfloat16),
           ((rows, f // 2), torch.uint8), ((rows, f // 32), torch.uint8), ((f, rows // 2), torch.uint8), ((f, rows // 32), torch.uint8))]
    got = gpu_lib.fp4_swiglu_producer_experts(dev(offsets), *map(dev, xq), dev(wc), dev(ws), mask, out=out)
    some = gpu_lib.fp4_swiglu_producer_experts(dev(offsets), *map(dev, xq), dev(wc), dev(ws), mask, emit_cols=False)
    assert some[4] is None and all(torch.equal(g, s) for g, s in zip(got[:4], some[:4]))
    bits = [host(t.view(torch.int16)) if t.dtype is torch.bfloat16 else host(t) for t in got]
    whole = d % 256 == 0
    for i in range(len(sizes)):
        lo, hi = offsets[i], offsets[i + 1]
        if lo == hi:
            continue
        want = [host(t) for t in gpu_lib.fp4_swiglu_producer(dev(xq[0][lo:hi]), dev(xq[1][lo:hi]), dev(wc[i]), dev(ws[i]), mask)]
        mine = [b[lo:hi] for b in bits[:4]] + [bits[4][:, lo // 2:hi // 2], bits[5][:, lo // 32:hi // 32]]
        if whole:
            assert all(np.array_equal(m, v) for m, v in zip(mine, want)), i
        else:                                            # another main loop: a and b within a bf16 step, h from them
            for m, v in zip(mine[:2], want[:2]):
                m64, v64 = F.bf16_bits_to_f64(m.view(np.uint16)), F.bf16_bits_to_f64(v.view(np.uint16))
                assert (np.abs(m64 - v64) <= 2 * H * np.abs(v64) + 1e-4).all()
            hq = [F.decode(m[2], m[3]) for m in (mine, want)]
            assert np.linalg.norm(hq[0] - hq[1]) <= 0.02 * np.linalg.norm(hq[1])
    tail = [b[offsets[-1]:] for b in bits[:4]] + [bits[4][:, offsets[-1] // 2:] & 0x77, bits[5][:, offsets[-1] // 32:]]
    assert all((b == 0).all() for b in tail)


FEW = [((1,), 16, 32), ((0, 2), 17, 64), ((1, 0, 0, 1), 33, 96), ((16, 17, 33), 48, 128), ((3,) * 70, 20, 160), ((15, 1), 512, 1024),
       ((40, 0, 5), 100, 2080), ((2, 2), 4100, 512), ((9, 64), 256, 4096), ((1, 1), 64, 14336), ((5, 20), 40, 8192), ((0, 0), 8, 64),
       ((9, 1, 0, 7, 8), 200, 9600), ((6, 2, 2, 1), 33, 14336), ((1, 0, 3), 17, 73248)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("align,extra", [(1, 0), (1, 3), (32, 0)])
@pytest.mark.parametrize("sizes,n,k", FEW)
def test_few(gpu_lib, sizes, n, k, align, extra, kind):
    offsets, rows = segments(sizes, align)
    rows += extra
    if rows == 0:
        return
    bits = synthetic.tensor((rows, k), seed=k, outlier_rate=0.002, outlier_scale=20.0)
    if kind == "bf16":
        x64, scales = F.bf16_bits_to_f64(bits), None
        x = torch.zeros((rows, k + 8), dtype=torch.bfloat16, device="cuda")[:, :k]
        x.copy_(dev(bits.view(np.int16)).view(torch.bfloat16))
    else:
        c, s = N.encode_e4m3(bits)
        x64, x, scales = N.decode_e4m3(c, s), dev(c), dev(s)
    w = codes((len(sizes), n, k), 2)
    ref, e = np.zeros((2, rows, n))
    for i in range(len(sizes)):
        at, wi = slice(offsets[i], offsets[i + 1]), F.decode(w[0][i], w[1][i])
        ref[at], e[at] = x64[at] @ wi.T, abs(x64[at]) @ abs(wi).T
    out = torch.full((rows, n + 3), 7.0, device="cuda")
    got = gpu_lib.fp4_matvec_experts(dev(offsets), x, *map(dev, w), x_scales=scales, c=out[:, :n])
    check(got, ref, e, k)
    assert (host(out)[:, n:] == 7).all() and (host(got)[offsets[-1]:] == 0).all()


FEW_GATED = [((1,), 8, 32), ((1,), 1, 32), ((0, 2, 1), 17, 96), ((16, 17, 33), 48, 128), ((2, 2), 1500, 4096), ((20, 3), 40, 8192),
             ((3,) * 66, 24, 544), ((9, 2, 0, 4), 40, 8192)]


def check_gate(got, want, x64, w13):
    """Two h of the same rows by different splits of the fp32 sums.  The sums a and
    b are each within 1e-5 sum |x w| of their values, so that two differ by twice
    that, which moves h by 1.1 |b| times a's and |silu(a)| times b's (silu' is below
    1.1).  They may then round to neighbouring bf16 values: d ln silu(a) / d ln a = 1
    + a (1 - sig(a)) lies within 1 + |a|, so that one step of a, 2 H of it, moves
    ln |h| by 2 H (1 + |a|) at most, a step of b and h's own by 2 H each."""
    f = len(w13) // 2
    a, b = x64 @ w13[:f].T, x64 @ w13[f:].T
    ea, eb = abs(x64) @ abs(w13[:f]).T, abs(x64) @ abs(w13[f:]).T
    tol = 2e-5 * (1.1 * abs(b) * ea + abs(A.value(a, A.SILU)) * eb + 2e-5 * ea * eb)
    got, want = host(got), host(want)
    steps = np.exp(2 * H * (3 + 1.01 * abs(a)))
    assert (np.abs(got - want) <= (steps - 1) * np.abs(want) + steps * tol + 2.0 ** -130).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,f,d", FEW_GATED)
def test_few_gated_rows_are_those_of_the_plain_call(gpu_lib, sizes, f, d, kind):
    """h of each row against fp4_swiglu_matvec on it."""
    offsets, rows = segments(sizes, 1)
    rows += 2
    bits = synthetic.tensor((rows, d), seed=d)
    x64, x, scales = F.bf16_bits_to_f64(bits), dev(bits.view(np.int16)).view(torch.bfloat16), None
    if kind == "e4m3":
        x64, (x, scales) = N.decode_e4m3(*N.encode_e4m3(bits)), map(dev, N.encode_e4m3(bits))
    w = [dev(t) for t in codes((len(sizes), 2 * f, d), 2)]
    got = gpu_lib.fp4_swiglu_matvec_experts(dev(offsets), x, *w, x_scales=scales)
    assert (host(got)[offsets[-1]:] == 0).all()
    for i in range(len(sizes)):
        for lo in range(offsets[i], offsets[i + 1], 64):
            at = slice(lo, min(lo + 64, offsets[i + 1]))
            want = gpu_lib.fp4_swiglu_matvec(x[at], w[0][i], w[1][i], x_scales=None if scales is None else scales[at])
            check_gate(got[at], want, x64[at], F.decode(host(w[0][i]), host(w[1][i])))


# rows a unit, output columns, K: scales one byte off a word, K of whole and part steps, x staged or not
UNALIGNED = [(1, 1, 64), (2, 40, 128), (3, 33, 160), (1, 70, 512), (2, 300, 544), (16, 64, 1024), (5, 200, 2080), (16, 48, 8192), (20, 33, 8224),
             (1, 9000, 512), (1, 16400, 1056)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("m,n,k", UNALIGNED)
def test_few_with_scales_off_words(gpu_lib, m, n, k, kind):
    """Weight scales that start one byte off a word (a view into a larger buffer), plain, gated and with an epilogue."""
    bits = synthetic.tensor((3 * m, k), seed=k)
    x64, x, scales = F.bf16_bits_to_f64(bits), dev(bits.view(np.int16)).view(torch.bfloat16), None
    if kind == "e4m3":
        c, s = N.encode_e4m3(bits)
        x64, x, scales = N.decode_e4m3(c, s), dev(c), dev(s)
    offsets = dev(np.array([0, m, m, 3 * m], np.int32))

    def off(a):
        buf = torch.zeros(a.size + 1, dtype=torch.uint8, device="cuda")
        buf[1:] = dev(a).reshape(-1)
        return buf[1:].reshape(a.shape)

    w = codes((3, n, k), 2)
    wd = [F.decode(w[0][i], w[1][i]) for i in range(3)]
    ref, e = np.zeros((2, 3 * m, n))
    for i, at in ((0, slice(0, m)), (2, slice(m, 3 * m))):
        ref[at], e[at] = x64[at] @ wd[i].T, abs(x64[at]) @ abs(wd[i]).T
    check(gpu_lib.fp4_matvec_experts(offsets, x, dev(w[0]), off(w[1]), x_scales=scales), ref, e, k)
    few = slice(0, m)
    got = gpu_lib.fp4_matvec_act(x[few], dev(w[0][0]), off(w[1][0]), x_scales=None if scales is None else scales[few], dtype=torch.float32)
    check(got, ref[few], e[few], k)
    w = codes((3, 2 * n, k), 3)
    want = gpu_lib.fp4_swiglu_matvec_experts(offsets, x, dev(w[0]), dev(w[1]), x_scales=scales)
    got = gpu_lib.fp4_swiglu_matvec_experts(offsets, x, dev(w[0]), off(w[1]), x_scales=scales)
    for i, at in ((0, slice(0, m)), (2, slice(m, 3 * m))):
        check_gate(got[at], want[at], x64[at], F.decode(w[0][i], w[1][i]))


# and items of four steps with scales off words, or ending in a part step
VARIANTS = SHAPES + [(3, 14336, 2048, 1), (2, 14337, 1952, 0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k,off", VARIANTS)
def test_few_row_variants(gpu_lib, m, n, k, off, kind):
    """The shapes that reach every variant of the plain few-row products, for the
    one with an epilogue and, up to sixteen rows, for one expert's rows."""
    bits = synthetic.tensor((m, k), seed=k)
    x64, x, scales = F.bf16_bits_to_f64(bits), dev(bits.view(np.int16)).view(torch.bfloat16), None
    if kind == "e4m3":
        c, s = N.encode_e4m3(bits)
        x64, x, scales = N.decode_e4m3(c, s), dev(c), dev(s)

    def at(a):
        buf = torch.zeros(a.size + off, dtype=torch.uint8, device="cuda")
        buf[off:] = dev(a).reshape(-1)
        return buf[off:].reshape(a.shape)

    w = codes((1, n, k), 2)
    W = torch.from_numpy(F.decode(w[0][0], w[1][0])).cuda()
    X = torch.from_numpy(np.ascontiguousarray(x64)).cuda()
    ref, e = host(X @ W.t()), host(X.abs() @ W.abs().t())
    wc, ws = dev(w[0]), at(w[1])
    check(gpu_lib.fp4_matvec_act(x, wc[0], ws[0], x_scales=scales, dtype=torch.float32), ref, e, k)
    if m > 16:
        return
    offsets = dev(np.array([0, m], np.int32))
    check(gpu_lib.fp4_matvec_experts(offsets, x, wc, ws, x_scales=scales), ref, e, k)
    w = codes((1, 2 * n, k), 3)
    wc, ws = dev(w[0]), at(w[1])
    got = gpu_lib.fp4_swiglu_matvec_experts(offsets, x, wc, ws, x_scales=scales)
    want = gpu_lib.fp4_swiglu_matvec(x, wc[0], ws[0], x_scales=scales)
    check_gate(got, want, x64, F.decode(w[0][0], w[1][0]))


@pytest.mark.parametrize("k", [96, 160, 1056, 2080])
def test_a_weight_row_does_not_reach_its_neighbours(gpu_lib, k):
    """Scale byte 255, which stands for no number, in one row of W: that column of
    C may hold anything, the others stay as they are."""
    n, bad = 40, [1, 17, 39]
    bits = synthetic.tensor((3, k), seed=k)
    x = dev(bits.view(np.int16)).view(torch.bfloat16)
    c, s = codes((1, n, k), 2)
    offsets = dev(np.array([0, 3], np.int32))
    broken = s.copy()
    broken[0, bad] = 255
    good = np.setdiff1d(np.arange(n), bad)

    def run(s):
        y = [gpu_lib.fp4_matvec_experts(offsets, x, dev(c), dev(s)), gpu_lib.fp4_matvec_act(x, dev(c[0]), dev(s[0]), dtype=torch.float32),
             gpu_lib.fp4_matvec(x, dev(c[0]), dev(s[0]))]
        return [host(v)[:, good] for v in y]

    for name, got, want in zip(("experts", "act", "plain"), run(broken), run(s)):
        assert np.array_equal(got, want), name


@pytest.mark.parametrize("n,k", [(32, 96), (64, 288), (256, 544)])
def test_rows_and_weights_do_not_reach_their_neighbours(gpu_lib, n, k):
    """The same of a row of A and of B in the long products."""
    sizes = (40, 0, 33)
    offsets, rows = segments(sizes, 1)
    a, b = codes((rows, k), 1), codes((len(sizes), n, k), 2)
    ab, bb = a[1].copy(), b[1].copy()
    ab[[0, 41, rows - 1]] = 255
    bb[0, [0, n - 1]], bb[2, 7] = 255, 255
    ok = np.zeros((rows, n), bool)
    ok[:40, 1:n - 1] = True
    ok[40:] = np.arange(n) != 7
    ok[[0, 41, rows - 1]] = False

    def run(sa, sb):
        got = [host(gpu_lib.fp4_gemm_experts(dev(offsets), dev(a[0]), dev(sa), dev(b[0]), dev(sb)))[ok]]
        y = host(gpu_lib.fp4_gemm_act(dev(a[0]), dev(sa), dev(b[0][0]), dev(sb[0]), dtype=torch.float32)[0])
        good = np.ones((rows, n), bool)
        good[[0, 41, rows - 1]], good[:, [0, n - 1]] = False, False
        return got + [y[good]]

    for got, want in zip(run(ab, bb), run(a[1], b[1])):
        assert np.isfinite(want).all() and np.array_equal(got, want)


@pytest.mark.parametrize("sizes", [(32, 64, 32), (96, 32, 0, 160, 224), (288, 32, 512)])
def test_tokens_do_not_reach_other_experts(gpu_lib, sizes):
    """Scale bytes that stand for no number in one expert's tokens (a NaN in its
    activations or gradients) leave the other experts' weight gradients as they are."""
    offsets, tokens = segments(sizes, 32)
    m, n = 64, 96
    pad = -tokens % 256
    a, b = codes((m, tokens + pad), 1), codes((n, tokens + pad), 2)
    for e in range(len(sizes)):
        at = slice(offsets[e] // 32, offsets[e + 1] // 32)
        sa, sb = a[1].copy(), b[1].copy()
        sa[:, at], sb[3, at] = 255, 255
        sa[:, tokens // 32:], sb[:, tokens // 32:] = 255, 255
        for dtype in (torch.float32, torch.bfloat16):
            want = host(gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), dev(a[0]), dev(a[1]), dev(b[0]), dev(b[1]), dtype=dtype))
            got = host(gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), dev(a[0]), dev(sa), dev(b[0]), dev(sb), dtype=dtype))
            others = [i for i in range(len(sizes)) if i != e]
            assert np.array_equal(got[others], want[others])


@pytest.mark.parametrize("k", [96, 288, 544])
def test_rows_and_weights_of_many_tiles_do_not_reach_their_neighbours(gpu_lib, k):
    sizes, n = (2400, 0, 800), 2080
    offsets, rows = segments(sizes, 1)
    a, b = codes((rows, k), 1), codes((len(sizes), n, k), 2)
    ab, bb = a[1].copy(), b[1].copy()
    broken = [0, 256, 2400, rows - 1]
    ab[broken] = 255
    bb[0, [0, n - 1]], bb[2, 7] = 255, 255
    ok = np.ones((rows, n), bool)
    ok[:2400, [0, n - 1]], ok[2400:, 7], ok[broken] = False, False, False
    good = np.ones((rows, n), bool)
    good[:, [0, n - 1]], good[broken] = False, False

    def run(sa, sb):
        ac, as_, bc, bs = dev(a[0]), dev(sa), dev(b[0]), dev(sb)
        return [host(gpu_lib.fp4_gemm_experts(dev(offsets), ac, as_, bc, bs))[ok],
                host(gpu_lib.fp4_gemm_act(ac, as_, bc[0], bs[0], dtype=torch.float32)[0])[good]]

    for got, want in zip(run(ab, bb), run(a[1], b[1])):
        assert np.isfinite(want).all() and np.array_equal(got, want)


def test_tokens_of_many_tiles_do_not_reach_other_experts(gpu_lib):
    sizes, m, n = (96, 32, 0, 160, 224), 1056, 1056
    offsets, tokens = segments(sizes, 32)
    a, b = codes((m, 512), 1), codes((n, 512), 2)
    want = host(gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), dev(a[0]), dev(a[1]), dev(b[0]), dev(b[1])))
    for e in range(len(sizes)):
        at = slice(offsets[e] // 32, offsets[e + 1] // 32)
        sa, sb = a[1].copy(), b[1].copy()
        sa[:, at], sb[3, at], sa[:, tokens // 32:] = 255, 255, 255
        got = host(gpu_lib.fp4_gemm_experts_wgrad(dev(offsets), dev(a[0]), dev(sa), dev(b[0]), dev(sb)))
        others = [i for i in range(len(sizes)) if i != e]
        assert np.array_equal(got[others], want[others])
