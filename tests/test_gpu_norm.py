"""GPU checks of dropout, the RMSNorm producer and its gradients against the
float64 oracle.

Exact: the mask, s, the codes of the emitted y.  With u = 2^-24 (half an fp32
step) and h = 2^-8 (half a bf16 step):
  rstd   the squares are summed by at most 32 fused steps a thread, 6 lane and
         16 wave additions, then divide, add, root, divide: 54/2 + 4 of u at most;
  y      rstd's, two products and the bf16 rounding;
  dsum   mean(g xh) carries the products' and 54 sums' u on mean |g xh|, the
         remaining five operations u each on the terms' magnitudes, then h;
  dgamma at most t/512 + 48 additions on sum |dy xh|, two product roundings.
"""

import numpy as np
import pytest
import torch

import synthetic
from oracle import formats as F
from oracle import norm as N
from oracle import quant as Q

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8
TINY = 2.0 ** -133                                       # the subnormal bf16 spacing


def dev16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def val(t):
    return F.bf16_bits_to_f64(bits(t))


def inputs(shape, seed, f32, std=1.0):
    b = synthetic.tensor(shape, std=std, seed=seed, outlier_rate=0.002, outlier_scale=20.0)
    x = F.bf16_bits_to_f64(b).astype(np.float32)
    if not f32:
        return x, dev16(b)
    x = (x * np.float32(1.0009765)).astype(np.float32)     # values with more bits than bf16 holds
    return x, torch.from_numpy(x).cuda()


SHAPES = [(1, 32), (17, 32), (3, 96), (5, 128), (7, 160), (4, 512), (2, 544), (3, 1024), (2, 1056), (2, 2048), (3, 2080),
          (2, 4096), (2, 4128), (1, 8192), (2, 8224), (1, 16384), (2, 16416), (1, 32768), (300, 64), (33, 4096)]


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("f32,res,p", [(False, True, 0.0), (True, True, 0.1), (False, False, 0.0), (True, False, 0.5)])
def test_producer(gpu_lib, t, d, f32, res, p):
    mx = gpu_lib
    x, xd = inputs((t, d), 1, f32)
    rb = synthetic.tensor((t, d), std=2.0, seed=2) if res else None
    gb = synthetic.bf16_bits((1 + 0.2 * np.random.default_rng(3).standard_normal(d)).astype(np.float32))
    if t > 2:                                            # a zero row and a row of one value
        x[1] = 0
        xd[1] = 0
        if res:
            rb[1] = 0
    seed, offset = 2 ** 35 + 11, 2 ** 32 + 5
    rd = None if rb is None else dev16(rb)
    s, rstd, y, codes, scales = mx.fp4_rmsnorm_producer(xd, dev16(gb), 1e-5, rd, p, seed, offset, mx.FP4_E4M3,
                                                        emit_y=True)
    sb = N.dropout_bits(x, p, seed, offset, rb)
    assert np.array_equal(bits(s), sb)
    r64, y64 = N.rmsnorm(F.bf16_bits_to_f64(sb), F.bf16_bits_to_f64(gb), 1e-5)
    assert (np.abs(host(rstd) - r64) <= 32 * U * r64).all()
    assert (np.abs(val(y) - y64) <= (H + 36 * U) * np.abs(y64) + TINY).all()
    yb = bits(y)
    for fmt, want in ((mx.FP4_E4M3, N.encode_e4m3(yb)), (mx.FP4_E2M1, Q.quantize_rows(yb))):
        # with neither the sum nor y emitted the codes stay the same bytes
        n, rstd2, none, c2, sc2 = mx.fp4_rmsnorm_producer(xd, dev16(gb), 1e-5, rd, p, seed, offset, fmt, emit_sum=False)
        assert n is None and none is None
        assert np.array_equal(host(rstd2), host(rstd))
        assert np.array_equal(host(c2), want[0]) and np.array_equal(host(sc2), want[1])
    assert np.array_equal(host(codes), N.encode_e4m3(yb)[0]) and np.array_equal(host(scales), N.encode_e4m3(yb)[1])


def test_e4m3_codes_of_every_bf16_value(gpu_lib):
    """s = 1 in every place and a vanishing eps make rstd = 1 and y = gamma."""
    mx = gpu_lib
    pos = np.arange(0, 0x7F80, dtype=np.uint16)
    pos = pos[: len(pos) // 32 * 32]
    rng = np.random.default_rng(5)
    for g in (pos, pos | np.uint16(0x8000), rng.permutation(pos), rng.permutation(pos) ^ np.uint16(0x8000)):
        x = dev16(np.full((1, len(g)), 0x3F80, np.uint16))
        _, rstd, y, codes, scales = mx.fp4_rmsnorm_producer(x, dev16(g), 1e-30, emit_y=True)
        assert host(rstd)[0] == 1.0 and np.array_equal(bits(y)[0], g)
        want = N.encode_e4m3(g[None])
        assert np.array_equal(host(scales), want[1])
        assert np.array_equal(host(codes), want[0])


def test_producer_strided_views_and_given_buffers(gpu_lib):
    mx = gpu_lib
    t, d = 5, 96
    for f32 in (False, True):
        x, xd = inputs((t, 160), 4, f32)
        rb = synthetic.tensor((t, 128), seed=5)
        gb = synthetic.bf16_bits(np.linspace(0.5, 1.5, d, dtype=np.float32))
        bufs = [torch.empty((t, d), dtype=torch.int16, device="cuda"), torch.empty(t, device="cuda"),
                torch.empty((t, d), dtype=torch.bfloat16, device="cuda"),
                torch.empty((t, d), dtype=torch.uint8, device="cuda"), torch.empty((t, d // 32), dtype=torch.uint8, device="cuda")]
        got = mx.fp4_rmsnorm_producer(xd[:, 32:32 + d], dev16(gb), 1e-5, dev16(rb)[:, 16:16 + d], 0.1, 3, 4, emit_y=True,
                                      out=bufs)
        assert all(a is b for a, b in zip(got, bufs))
        sb = N.dropout_bits(x[:, 32:32 + d], 0.1, 3, 4, rb[:, 16:16 + d])
        assert np.array_equal(bits(got[0]), sb)
        assert np.array_equal(host(got[3]), N.encode_e4m3(bits(got[2]))[0])


BWD_SHAPES = [(1, 32), (17, 32), (513, 64), (1100, 160), (3, 544), (5, 1056), (70, 4096), (520, 1056), (3, 8224), (2, 16416),
              (2, 32768), (600, 128)]


@pytest.mark.parametrize("t,d", BWD_SHAPES)
@pytest.mark.parametrize("f32,with_ds,p", [(True, True, 0.1), (False, False, 0.0), (True, False, 0.5), (False, True, 0.0)])
def test_backward(gpu_lib, t, d, f32, with_ds, p):
    mx = gpu_lib
    dy, dyd = inputs((t, d), 7, f32, std=1e-3)
    sb = synthetic.tensor((t, d), std=2.0, seed=8, outlier_rate=0.001, outlier_scale=20.0)
    if t > 2:
        sb[2] = 0                                        # rstd = 1 / sqrt(eps)
    gb = synthetic.bf16_bits((1 + 0.2 * np.random.default_rng(9).standard_normal(d)).astype(np.float32))
    db = synthetic.tensor((t, d), std=1e-3, seed=10) if with_ds else None
    s64, g64 = F.bf16_bits_to_f64(sb), F.bf16_bits_to_f64(gb)
    rstd = N.rmsnorm(s64, g64, 1e-5)[0].astype(np.float32)
    seed, offset = 77, 2 ** 40 + 9
    dsum, dx, dgamma = mx.fp4_rmsnorm_backward(dyd, dev16(sb), torch.from_numpy(rstd).cuda(), dev16(gb),
                                               None if db is None else dev16(db), p, seed, offset)
    r = rstd.astype(np.float64)
    dy64, ds64 = dy.astype(np.float64), None if db is None else F.bf16_bits_to_f64(db)
    want, want_g = N.rmsnorm_backward(dy64, s64, r, g64, ds64)
    xh, g = s64 * r[:, None], dy64 * g64
    size = r[:, None] * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    size = size + (0 if ds64 is None else np.abs(ds64))
    near = lambda got, ref, m: (np.abs(got - ref) <= H * np.abs(ref) + 64 * U * m + TINY).all()  # noqa: E731
    assert near(val(dsum), want, size)
    if p > 0:
        keep, scale = N.keep_mask(t, d, p, seed, offset), float(N.keep_scale(p))
        got = val(dx)
        assert (got[~keep] == 0).all()
        assert near(got, np.where(keep, want * scale, 0.0), scale * size)
    else:
        assert dx is dsum
    bound = (t / 512 + 64) * U * np.abs(dy64 * xh).sum(axis=0)
    assert (np.abs(host(dgamma) - want_g) <= bound + 2.0 ** -149).all()
    # accumulation adds the same sum to what is there
    first = host(dgamma).copy()
    _, _, again = mx.fp4_rmsnorm_backward(dyd, dev16(sb), torch.from_numpy(rstd).cuda(), dev16(gb),
                                          None if db is None else dev16(db), p, seed, offset, accumulate=True,
                                          out=(None, None, dgamma))
    assert again is dgamma
    assert (np.abs(host(again) - 2 * want_g) <= 2 * bound + 20 * U * np.abs(first) + 2.0 ** -148).all()


def test_backward_of_no_rows(gpu_lib):
    mx = gpu_lib
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((64,), 3.0, device="cuda")
    mx.fp4_rmsnorm_backward(z, z, torch.empty(0, device="cuda"), g, accumulate=True, out=(None, None, out))
    assert (host(out) == 3).all()
    mx.fp4_rmsnorm_backward(z, z, torch.empty(0, device="cuda"), g, out=(None, None, out))
    assert (host(out) == 0).all()
    s, rstd, y, codes, scales = mx.fp4_rmsnorm_producer(z, g)
    assert s.shape == (0, 64) and codes.shape == (0, 64) and scales.shape == (0, 2)


def test_backward_strided_views(gpu_lib):
    mx = gpu_lib
    t, d = 9, 64
    for f32 in (True, False):
        dy, dyd = inputs((t, 96), 11, f32)
        sb, db = synthetic.tensor((t, 128), seed=12), synthetic.tensor((t, 80), seed=13)
        gb = synthetic.bf16_bits(np.linspace(0.5, 1.5, d, dtype=np.float32))
        rstd = np.linspace(0.5, 2, t, dtype=np.float32)
        got = mx.fp4_rmsnorm_backward(dyd[:, 32:], dev16(sb)[:, 8:8 + d], torch.from_numpy(rstd).cuda(), dev16(gb),
                                      dev16(db)[:, 16:])
        want = mx.fp4_rmsnorm_backward(dyd[:, 32:].contiguous(), dev16(sb)[:, 8:8 + d].contiguous(),
                                       torch.from_numpy(rstd).cuda(), dev16(gb), dev16(db)[:, 16:].contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (1, 8), (3, 9), (5, 32), (2, 4099), (129, 65), (64, 1000), (4097, 3)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("res,p", [(False, 0.1), (True, 0.25), (True, 0.0), (False, 1.0)])
def test_dropout(gpu_lib, rows, cols, f32, res, p):
    mx = gpu_lib
    x, xd = inputs((rows, cols), 21, f32)
    rb = synthetic.tensor((rows, cols), seed=22) if res else None
    seed, offset = 2 ** 63 + 3, 2 ** 63 + 9
    want = N.dropout_bits(x, p, seed, offset, rb)
    # rows as they lie (odd pitches: element by element), and padded to a pitch of eight (wide loads)
    pad = lambda t: torch.nn.functional.pad(t, (0, -cols % 8), value=7.0)[:, :cols]  # noqa: E731
    for put in (lambda t: t, pad):
        got = mx.fp4_dropout(put(xd), p, seed, offset, None if rb is None else put(dev16(rb)))
        assert np.array_equal(bits(got), want)
    # an output inside a larger tensor: what lies around it stays
    out = torch.full((rows + 1, cols + 3), -5.0, dtype=torch.bfloat16, device="cuda")
    mx.fp4_dropout(xd, p, seed, offset, None if rb is None else dev16(rb), out=out[:rows, :cols])
    o = val(out)
    assert np.array_equal(bits(out[:rows, :cols]), want)
    assert (o[rows] == -5).all() and (o[:, cols:] == -5).all()


def test_dropout_of_infinities_and_nan(gpu_lib):
    mx = gpu_lib
    x = torch.ones((8, 72), device="cuda")
    keep = torch.from_numpy(N.keep_mask(8, 72, 0.5, 1, 1)).cuda()
    x[~keep] = float("nan")
    x[0, :] = torch.where(keep[0], x[0], float("inf"))
    for v in (x, x.bfloat16()):
        out = mx.fp4_dropout(v, 0.5, 1, 1)
        assert torch.equal(out, torch.where(keep, 2.0, 0.0).bfloat16())
    kept = torch.where(keep, float("nan"), 1.0)
    assert torch.equal(mx.fp4_dropout(kept, 0.5, 1, 1).isnan(), keep)


def test_dropout_past_32_bit_offsets(gpu_lib):
    mx = gpu_lib
    rows, cols = 65600, 65544                            # 4.3e9 elements, 8.6 GB
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    out = mx.fp4_dropout(x, 0.25, 5, 6)
    want_scale = float(synthetic_bf16(N.keep_scale(0.25)))
    for r in (0, 1, 32766, 65535, 65599):
        # the mask of one row alone: the oracle's indexes of that row
        keep = row_mask(r, cols, 0.25, 5, 6)
        assert np.array_equal(val(out[r:r + 1])[0], np.where(keep, want_scale, 0.0))
    del x, out
    torch.cuda.empty_cache()


def synthetic_bf16(v):
    return F.bf16_bits_to_f64(N.f32_to_bf16_rne(np.float32(v)))


def row_mask(r, cols, p, seed, offset):
    from oracle import philox as P
    i = np.uint64(r) * np.uint64(8 * -(-cols // 8)) + np.arange(cols, dtype=np.uint64)
    word = P.draws(seed, offset, ((i >> np.uint64(3)) << np.uint64(2)) + ((i >> np.uint64(1)) & np.uint64(3)))
    return np.where(i & np.uint64(1), word >> np.uint64(16), word & np.uint64(0xFFFF)) >= N.threshold(p)


def test_refusals_of_the_binding(gpu_lib):
    mx = gpu_lib
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = torch.ones(4, device="cuda")
    bad = [
        lambda: mx.fp4_rmsnorm_producer(x.cpu(), g), lambda: mx.fp4_rmsnorm_producer(x.double(), g),
        lambda: mx.fp4_rmsnorm_producer(x.t(), g), lambda: mx.fp4_rmsnorm_producer(x[0], g),
        lambda: mx.fp4_rmsnorm_producer(x, g[:32]), lambda: mx.fp4_rmsnorm_producer(x, g.float()),
        lambda: mx.fp4_rmsnorm_producer(x, g, residual=x[:2]), lambda: mx.fp4_rmsnorm_producer(x, g, residual=x.float()),
        lambda: mx.fp4_rmsnorm_producer(x, g, 0.0), lambda: mx.fp4_rmsnorm_producer(x, g, p=1.5),
        lambda: mx.fp4_rmsnorm_producer(x[:, :48], g[:48]), lambda: mx.fp4_rmsnorm_producer(x, g, fmt=3),
        lambda: mx.fp4_rmsnorm_producer(x[:1].expand(4, 64), g),
        lambda: mx.fp4_rmsnorm_producer(x, g, out=[None, None, None, x, None]),
        lambda: mx.fp4_rmsnorm_backward(x, x[:2], r, g), lambda: mx.fp4_rmsnorm_backward(x, x, r[:3], g),
        lambda: mx.fp4_rmsnorm_backward(x, x, r.double(), g), lambda: mx.fp4_rmsnorm_backward(x, x, r, g, accumulate=True),
        lambda: mx.fp4_rmsnorm_backward(x, x.float(), r, g), lambda: mx.fp4_rmsnorm_backward(x, x, r, g, ds=x.float()),
        lambda: mx.fp4_dropout(x, -0.1), lambda: mx.fp4_dropout(x, float("nan")), lambda: mx.fp4_dropout(x.half(), 0.1),
        lambda: mx.fp4_dropout(x, 0.1, residual=x[:, :32]), lambda: mx.fp4_dropout(x, 0.1, out=x.float()),
        lambda: mx.fp4_dropout(x, 0.1, out=x[:1].expand(4, 64)),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(mx.Fp4Error):
            f()
            pytest.fail(f"call {k} was not refused")


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(gpu_lib, seed):
    """Shapes drawn over the whole range: the sum and the codes exactly, y and
    the gradients in the 2-norm (their roundings, and 2^-16 for the fp32 sums)."""
    mx, rng = gpu_lib, np.random.default_rng(500 + seed)
    log = lambda lo, hi: int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))  # noqa: E731
    t, d, p, f32 = log(1, 1500), 32 * log(1, 512), (0.0, 0.1, 0.6)[seed % 3], seed % 2 == 1
    t = max(1, min(t, (1 << 21) // d))
    x, xd = inputs((t, d), 600 + seed, f32)
    rb = synthetic.tensor((t, d), std=1.0, seed=700 + seed) if seed % 4 else None
    gb = synthetic.bf16_bits((1 + 0.2 * rng.standard_normal(d)).astype(np.float32))
    sb = N.dropout_bits(x, p, seed, seed, rb)
    s, rstd, y, codes, scales = mx.fp4_rmsnorm_producer(xd, dev16(gb), 1e-5, None if rb is None else dev16(rb), p, seed,
                                                        seed, emit_y=True)
    assert np.array_equal(bits(s), sb)
    want = N.encode_e4m3(bits(y))
    assert np.array_equal(host(codes), want[0]) and np.array_equal(host(scales), want[1])
    s64, g64 = F.bf16_bits_to_f64(sb), F.bf16_bits_to_f64(gb)
    near = lambda got, ref, tol: np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref)  # noqa: E731
    r64, y64 = N.rmsnorm(s64, g64, 1e-5)
    assert near(host(rstd), r64, 2.0 ** -18) and near(val(y), y64, H)
    db = None if rb is None else dev16(rb)
    dsum, dx, dgamma = mx.fp4_rmsnorm_backward(xd, s, rstd, dev16(gb), db, p, seed, seed)
    ds, dg = N.rmsnorm_backward(x.astype(np.float64), s64, host(rstd).astype(np.float64), g64,
                                None if rb is None else F.bf16_bits_to_f64(rb))
    assert near(val(dsum), ds, H + 2.0 ** -16) and near(host(dgamma), dg, 2.0 ** -16)
    keep, sc = N.keep_mask(t, d, p, seed, seed), float(N.keep_scale(p))
    assert near(val(dx), np.where(keep, ds * sc, 0.0), H + 2.0 ** -16)


def test_everything_dropped(gpu_lib):
    """p = 1: s is the residual (or zero), nothing flows back to x."""
    mx, t, d = gpu_lib, 6, 96
    x, xd = inputs((t, d), 31, True)
    rb = synthetic.tensor((t, d), seed=32)
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    s, rstd, *_ = mx.fp4_rmsnorm_producer(xd, g, 1e-5, dev16(rb), 1.0, 3, 4)
    assert torch.equal(s, dev16(rb))
    dsum, dx, _ = mx.fp4_rmsnorm_backward(xd, s, rstd, g, p=1.0, seed=3, offset=4)
    assert (val(dx) == 0).all() and (val(dsum) != 0).any()
    s, rstd, y, codes, scales = mx.fp4_rmsnorm_producer(xd, g, 1e-5, None, 1.0, 3, 4, emit_y=True)
    assert (val(s) == 0).all() and (val(y) == 0).all() and (host(codes) == 0).all() and (host(scales) == 0).all()


def test_a_probability_below_the_resolution_drops_nothing(gpu_lib):
    mx = gpu_lib
    x, xd = inputs((4, 64), 33, False)
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for p in (0.0, 1e-6, 7.62939453125e-06 * 0.999):
        assert torch.equal(mx.fp4_dropout(xd, p, 1, 2), xd)
        s, rstd, *_ = mx.fp4_rmsnorm_producer(xd, g, p=p, seed=1, offset=2)
        assert torch.equal(s, xd)
        dsum, dx, _ = mx.fp4_rmsnorm_backward(xd, s, rstd, g, p=p, seed=1, offset=2)
        assert dx is dsum
    # 2^-17 rounds up to one part in 65536
    dsum, dx, _ = mx.fp4_rmsnorm_backward(xd, s, rstd, g, p=2.0 ** -17, seed=1, offset=2)
    assert dx is not dsum


def test_bit_patterns_flags_and_given_gradients(gpu_lib):
    """16-bit integer tensors hold the same values; every output can be left
    out or given; the outputs that are made do not depend on which."""
    mx, t, d = gpu_lib, 7, 160
    x, xd = inputs((t, d), 34, False)
    gb = synthetic.bf16_bits(np.linspace(0.5, 1.5, d, dtype=np.float32))
    i16 = lambda v: v.view(torch.int16)  # noqa: E731
    full = mx.fp4_rmsnorm_producer(xd, dev16(gb), 1e-5, xd, emit_y=True)
    same = mx.fp4_rmsnorm_producer(i16(xd), i16(dev16(gb)), 1e-5, i16(xd), emit_y=True)
    assert all(torch.equal(a, b) for a, b in zip(full, same))
    for es in (False, True):
        for ey in (False, True):
            for ec in (False, True):
                got = mx.fp4_rmsnorm_producer(xd, dev16(gb), 1e-5, xd, emit_sum=es, emit_y=ey, emit_codes=ec)
                assert [v is not None for v in got] == [es, True, ey, ec, ec]
                assert all(v is None or torch.equal(v, w) for v, w in zip(got, full))
    want = mx.fp4_rmsnorm_backward(xd, full[0], full[1], dev16(gb), xd, 0.3, 5, 6)
    bufs = (torch.empty((t, d), dtype=torch.int16, device="cuda"), torch.empty_like(xd), torch.empty(d, device="cuda"))
    got = mx.fp4_rmsnorm_backward(i16(xd), full[0], full[1], dev16(gb), xd, 0.3, 5, 6, out=bufs)
    assert all(a is b for a, b in zip(got, bufs))
    assert torch.equal(got[0].view(torch.bfloat16), want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("rows,cols,pitch", [(5, 64, 64), (3, 33, 40), (2, 4099, 4099), (1030, 40, 48)])
def test_dropout_in_place(gpu_lib, rows, cols, pitch):
    """out may be x or the residual; the columns behind stay."""
    mx = gpu_lib
    xb, rb = synthetic.tensor((rows, pitch), seed=41), synthetic.tensor((rows, pitch), seed=42)
    x, r = dev16(xb), dev16(rb)
    want = mx.fp4_dropout(x[:, :cols], 0.25, 7, 8, residual=r[:, :cols])
    for place in (0, 1):
        bufs = [dev16(xb), dev16(rb)]
        mx.fp4_dropout(bufs[0][:, :cols], 0.25, 7, 8, residual=bufs[1][:, :cols], out=bufs[place][:, :cols])
        assert torch.equal(bufs[place][:, :cols], want)
        assert torch.equal(bufs[place][:, cols:], (x, r)[place][:, cols:])


@pytest.mark.parametrize("t,d", [(1, 32), (17, 96), (5, 544), (300, 4096), (3, 8224), (2, 32768)])
def test_the_sum_takes_the_residuals_place(gpu_lib, t, d):
    mx = gpu_lib
    x, xd = inputs((t, d), 43, True)
    rb = synthetic.tensor((t, d), seed=44)
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    for p in (0.0, 0.2):
        want = mx.fp4_rmsnorm_producer(xd, g, 1e-5, dev16(rb), p, 3, 4, emit_y=True)
        res = dev16(rb)
        got = mx.fp4_rmsnorm_producer(xd, g, 1e-5, res, p, 3, 4, emit_y=True, out=(res, None, None, None, None))
        assert got[0] is res and all(torch.equal(a, b) for a, b in zip(got, want))
