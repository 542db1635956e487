"""GPU checks of the tokens sorted by expert: the order and the gathered rows
exactly, the weighted sum and its gradients against float64 within their fp32
sums and one rounding to bf16."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import experts as X
from oracle import formats as F
from oracle import norm as N
from oracle import quant as Q

pytestmark = pytest.mark.gpu
H, U = 2.0 ** -8, 2.0 ** -24                             # half a step of bf16 and of fp32


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(bits):
    return dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()


def choices(t, k, e, seed, spread="even"):
    """[t][k] experts: even, all on one, or with slots that are not routed."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, e, (t, k))
    if spread == "one":
        ids[:] = e - 1
    if spread == "holes":
        ids[rng.random((t, k)) < 0.3] = -1
        ids[rng.random((t, k)) < 0.1] = e + 5
        if t > 3:
            ids[1] = np.iinfo(np.int32).max
            ids[2] = np.iinfo(np.int32).min
    return ids


SORTS = [(0, 1, 1), (1, 1, 1), (1, 2, 8), (2, 8, 64), (63, 1, 3), (64, 1, 64), (65, 3, 65), (511, 2, 1024), (1000, 8, 160),
         (1024, 8, 64), (1025, 8, 64), (2731, 3, 7), (8192, 2, 8), (16384, 8, 256), (40000, 1, 1000), (131072, 8, 64)]


@pytest.mark.parametrize("spread", ["even", "one", "holes"])
@pytest.mark.parametrize("align", [1, 32, 256])
@pytest.mark.parametrize("t,k,e", SORTS)
def test_sort(gpu_lib, t, k, e, align, spread):
    ids = choices(t, k, e, t + k, spread)
    for dtype in (np.int32, np.int64):
        offsets, slots, rows = gpu_lib.fp4_expert_sort(dev(ids.astype(dtype)), e, align)
        want = X.sort(ids, e, align)
        assert np.array_equal(host(offsets), want[0])
        assert np.array_equal(host(slots), want[1])
        assert np.array_equal(host(rows), want[2])


def test_sort_takes_ids_past_32_bits_for_none(gpu_lib):
    ids = np.array([[0, 1 << 32], [(1 << 32) + 1, 1], [-(1 << 40), 2]], np.int64)
    got = gpu_lib.fp4_expert_sort(dev(ids), 3, 1)
    assert all(np.array_equal(host(g), w) for g, w in zip(got, X.sort(ids, 3, 1)))


def test_sort_into_longer_buffers(gpu_lib):
    ids = choices(50, 2, 6, 1)
    out = (torch.full((7,), 9, dtype=torch.int32, device="cuda"), torch.full((700,), 9, dtype=torch.int32, device="cuda"),
           torch.full((50, 2), 9, dtype=torch.int32, device="cuda"))
    got = gpu_lib.fp4_expert_sort(dev(ids), 6, 32, out=out)
    want = X.sort(ids, 6, 32, rows=700)
    assert all(g is o and np.array_equal(host(g), w) for g, o, w in zip(got, out, want))


GATHERS = [(1, 1, 1, 32), (1, 2, 8, 4096), (9, 2, 4, 64), (33, 3, 5, 96), (40, 2, 7, 128), (65, 8, 64, 160), (100, 1, 9, 1056),
           (130, 4, 16, 2048), (257, 2, 8, 2080), (17, 2, 3, 8192)]


@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("t,k,e,d", GATHERS)
def test_gather(gpu_lib, t, k, e, d, align):
    x = synthetic.tensor((t, d + 8), seed=d, outlier_rate=0.01, outlier_scale=20.0)[:, :d]   # rows at a pitch
    x[0, :32] = 0
    _, slots, _ = X.sort(choices(t, k, e, d, "holes"), e, align)
    want = X.gather(x, slots, k)
    xt = bf16(np.pad(x, ((0, 0), (0, 8))))[:, :d]
    for fmt, codec in ((gpu_lib.FP4_E2M1, Q.quantize_rows), (gpu_lib.FP4_E4M3, N.encode_e4m3)):
        xs, codes, scales = gpu_lib.fp4_expert_gather(xt, dev(slots), k, fmt=fmt)
        assert np.array_equal(host(xs.view(torch.int16)).view(np.uint16), want)
        wc, ws = codec(want) if len(slots) else (np.zeros((0, 1)), np.zeros((0, 1)))
        if len(slots):
            assert np.array_equal(host(codes), wc) and np.array_equal(host(scales), ws)
        only = gpu_lib.fp4_expert_gather(xt, dev(slots), k, fmt=fmt, emit_x=False)
        assert only[0] is None and torch.equal(only[1], codes) and torch.equal(only[2], scales)
    assert torch.equal(gpu_lib.fp4_expert_gather(xt, dev(slots), k, emit_codes=False)[0], xs)


def test_gather_takes_slots_of_no_token_for_padding(gpu_lib):
    x = synthetic.tensor((4, 64), seed=1)
    slots = np.array([0, 7, 8, -1, -5, 2 ** 31 - 1, -2 ** 31, 3], np.int32)         # 4 tokens with 2 slots each
    xs, _, _ = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), 2)
    want = X.gather(x, np.where((slots >= 0) & (slots < 8), slots, -1), 2)
    assert np.array_equal(host(xs.view(torch.int16)).view(np.uint16), want)


MANY_ROWS = [(2500, 6, 40, 2080, 32), (4100, 2, 8, 4160, 1), (450, 70, 90, 1024, 32)]


@pytest.mark.parametrize("t,k,e,d,align", MANY_ROWS)
def test_gather_of_many_rows(gpu_lib, t, k, e, d, align):
    """Past the size from which the rows go out token by token: the same bytes, rows without a token zero."""
    x = synthetic.tensor((t, d), seed=d)
    _, slots, _ = X.sort(choices(t, k, e, d, "holes"), e, align)
    assert gpu_lib.load().fp4_expert_gather_workspace(t, k, d, len(slots)) == 4 * t * k
    slots[-3:] = slots[0], -7, t * k                       # a slot twice, and two that are none
    want = X.gather(x, np.where((slots >= 0) & (slots < t * k), slots, -1), k)
    some = np.random.default_rng(0).choice(len(slots), 500)
    some = np.concatenate((some, [0, len(slots) - 3, len(slots) - 2, len(slots) - 1]))
    for fmt, codec in ((gpu_lib.FP4_E2M1, Q.quantize_rows), (gpu_lib.FP4_E4M3, N.encode_e4m3)):
        xs, codes, scales = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), k, fmt=fmt)
        assert np.array_equal(host(xs.view(torch.int16)).view(np.uint16), want)
        wc, ws = codec(want[some])
        assert np.array_equal(host(codes)[some], wc) and np.array_equal(host(scales)[some], ws)
        rest = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), k, fmt=fmt, emit_x=False)
        assert torch.equal(rest[1], codes) and torch.equal(rest[2], scales)


def parts(t, k, e, d, align, seed, zf32, spread="holes"):
    """Plan and tensors: (slots, where, z float64, z, weights)."""
    _, slots, where = X.sort(choices(t, k, e, seed, spread), e, align)
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(len(slots), d)).astype(np.float32)
    zt = dev(z) if zf32 else dev(z).bfloat16()
    return slots, where, host(zt).astype(np.float64), zt, rng.random((t, k)).astype(np.float32)


COMBINES = [(1, 1, 1, 32), (1, 2, 8, 4096), (9, 2, 8, 4096), (9, 8, 64, 64), (33, 3, 5, 96), (100, 5, 9, 1056), (200, 4, 16, 512),
            (63, 12, 20, 160), (31, 2, 3, 8192)]


@pytest.mark.parametrize("zf32", [False, True])
@pytest.mark.parametrize("align", [1, 32])
@pytest.mark.parametrize("t,k,e,d", COMBINES)
def test_combine(gpu_lib, t, k, e, d, align, zf32):
    slots, where, z64, z, w = parts(t, k, e, d, align, d + t, zf32)
    pad = torch.zeros((z.shape[0], d + 8), dtype=z.dtype, device="cuda")           # rows at a pitch
    pad[:, :d] = z
    res = np.random.default_rng(1).normal(size=(t, d)).astype(np.float32)
    rt = dev(res).bfloat16()
    for weights, residual in ((w, None), (None, None), (w, rt), (None, rt)):
        got = gpu_lib.fp4_expert_combine(pad[:, :d], dev(where), None if weights is None else dev(weights), residual=residual)
        want, mag = X.combine(z64, where, weights, None if residual is None else host(residual).astype(np.float64))
        # k fused steps and one addition in fp32, then one rounding
        tol = (k + 1) * U * mag
        assert (np.abs(host(got) - want) <= tol + H * (np.abs(want) + tol)).all()


def test_combine_onto_the_residual(gpu_lib):
    _, where, _, z, w = parts(20, 2, 4, 96, 1, 5, True)
    res = torch.randn(20, 96, device="cuda").bfloat16()
    want = gpu_lib.fp4_expert_combine(z, dev(where), dev(w), residual=res)
    out = gpu_lib.fp4_expert_combine(z, dev(where), dev(w), residual=res, out=res)
    assert out is res and torch.equal(res, want)


def test_an_unrouted_choice_leaves_no_trace(gpu_lib):
    where = np.array([[1, -1], [-1, -1], [3, 0], [9, 2]], np.int32)                 # 9: past the rows
    z = np.array([[1.0], [2], [3], [4]], np.float32) * np.ones((1, 32), np.float32)
    w = np.array([[0.5, np.nan], [np.inf, np.nan], [1, 1], [np.nan, 2]], np.float32)
    got = host(gpu_lib.fp4_expert_combine(dev(z), dev(where), dev(w)))
    assert (got == np.array([[1.0], [0], [5], [6]])).all()
    zz = z.copy()
    zz[0] = np.nan                                         # row 0 is read by no token below
    got = host(gpu_lib.fp4_expert_combine(dev(zz), dev(where[:2]), dev(w[:2])))
    assert (got == np.array([[1.0], [0]])).all()


@pytest.mark.parametrize("zf32", [False, True])
@pytest.mark.parametrize("dyf32", [False, True])
@pytest.mark.parametrize("t,k,e,d,align", [(*c, a) for c in COMBINES for a in (1, 32)])
def test_combine_backward(gpu_lib, t, k, e, d, align, dyf32, zf32):
    slots, where, z64, z, w = parts(t, k, e, d, align, d + t, zf32)
    dy = np.random.default_rng(2).normal(size=(t, d)).astype(np.float32)
    dyt = dev(dy) if dyf32 else dev(dy).bfloat16()
    dz = torch.full(z.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got_dz, got_dw = gpu_lib.fp4_expert_combine_backward(dyt, z, dev(slots), dev(where), dev(w), dz=dz)
    want_dz, want_dw, mag = X.combine_backward(host(dyt).astype(np.float64), z64, where, w)
    # one fp32 product, one rounding; fp32 sums of at most 8 ceil(d / 512) fused steps a lane and six additions
    assert (np.abs(host(got_dz) - want_dz) <= (H + 2 * U) * np.abs(want_dz)).all()
    assert (np.abs(host(got_dw) - want_dw) <= (8 * -(-d // 512) + 7) * U * mag).all()
    assert (host(got_dz)[slots < 0] == 0).all() and (host(got_dw)[where < 0] == 0).all()


def test_the_gradient_of_the_gather(gpu_lib):
    """combine without weights of a gradient in sorted order is the transpose of the gather."""
    t, k, e, d = 40, 3, 6, 64
    slots, where, z64, z, _ = parts(t, k, e, d, 32, 9, True)
    x = synthetic.tensor((t, d), seed=4)
    x64 = F.bf16_bits_to_f64(x)
    xs, _, _ = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), k, emit_codes=False)
    live = slots >= 0
    dx = host(gpu_lib.fp4_expert_combine(z, dev(where))).astype(np.float64)
    left, right = (host(xs).astype(np.float64) * z64)[live].sum(), (x64 * dx).sum()
    assert abs(left - right) <= (H + 4 * U) * (np.abs(x64) * X.combine(np.abs(z64), where)[0]).sum()


def test_no_tokens_and_no_rows(gpu_lib):
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    offsets, slots, rows = gpu_lib.fp4_expert_sort(ids, 4, 32)
    assert host(offsets).tolist() == [0] * 5 and slots.numel() == 0 and rows.shape == (0, 2)
    xs, codes, scales = gpu_lib.fp4_expert_gather(torch.zeros((0, 64), device="cuda").bfloat16(), slots, 2)
    assert xs.shape == (0, 64) and codes.shape == (0, 32) and scales.shape == (0, 2)
    # nothing routed: every row of the buffers is padding, every sum empty
    ids = torch.full((3, 2), -1, dtype=torch.int64, device="cuda")
    for align in (1, 32):
        offsets, slots, rows = gpu_lib.fp4_expert_sort(ids, 4, align)
        assert host(offsets).tolist() == [0] * 5 and (host(slots) == -1).all() and (host(rows) == -1).all()
        x = torch.randn(3, 64, device="cuda").bfloat16()
        xs, _, _ = gpu_lib.fp4_expert_gather(x, slots, 2)
        assert (host(xs) == 0).all()
        assert (host(gpu_lib.fp4_expert_combine(xs, rows, torch.ones((3, 2), device="cuda"))) == 0).all()
        assert torch.equal(gpu_lib.fp4_expert_combine(xs, rows, None, residual=x), x)
    none = torch.zeros((0, 64), device="cuda").bfloat16()
    assert (host(gpu_lib.fp4_expert_combine(none, rows, None)) == 0).all()
    dz, dw = gpu_lib.fp4_expert_combine_backward(x, none, slots[:0], rows, torch.ones((3, 2), device="cuda"))
    assert dz.shape == (0, 64) and (host(dw) == 0).all()
