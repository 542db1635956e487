"""The expert and epilogue calls in runs, as a layer uses them: one training step
of a gated layer of experts with its gradients, a decoded token through it, an
ungated FFN with the epilogue and its gradients; captured in a graph, on another
stream, and with no trace of what the buffers held."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import act as A
from oracle import experts as X
from oracle import formats as F
from oracle import quant as Q

pytestmark = pytest.mark.gpu
H = 2.0 ** -8


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(bits):
    return dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype is torch.bfloat16 else t.cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def close(got, want, tol):
    return np.linalg.norm(got - want) <= tol * np.linalg.norm(want)


class Layer:
    """A layer of E gated experts, D wide with F hidden columns: W1 and W3 stacked, W2."""

    def __init__(self, mx, E, D, Fh):
        self.mx, self.E, self.D, self.F = mx, E, D, Fh
        w13 = [Q.quantize_w2d32(synthetic.tensor((2 * Fh, D), std=0.1, seed=20 + e), 0.87) for e in range(E)]
        w2 = [Q.quantize_w2d32(synthetic.tensor((D, Fh), std=0.1, seed=60 + e), 0.87) for e in range(E)]
        stack = lambda ws, i: dev(np.stack([w[i] for w in ws]))  # noqa: E731
        self.w13, self.w2 = [stack(w13, i) for i in range(4)], [stack(w2, i) for i in range(4)]
        # the column layouts of W1 and W3 apart, for dX = dA W1 + dB W3
        self.w1c = [self.w13[2][:, :, :Fh // 2].contiguous(), self.w13[3][:, :, :Fh // 32].contiguous()]
        self.w3c = [self.w13[2][:, :, Fh // 2:].contiguous(), self.w13[3][:, :, Fh // 32:].contiguous()]
        self.mask = mx.fp4_sign_mask_from_seed(5)

    def step(self, x, ids, weights, res, dy):
        """Forwards and backwards; everything that a trainer would keep."""
        mx, E, mask, k = self.mx, self.E, self.mask, ids.shape[1]
        off, slots, rows = mx.fp4_expert_sort(ids, E, 32)
        xs, xc, xsc = mx.fp4_expert_gather(x, slots, k)
        xt = mx.fp4_quantize_cols(xs, 32, mask)
        a, b, hc, hs, htc, hts = mx.fp4_swiglu_producer_experts(off, xc, xsc, *self.w13[:2], mask)
        z = mx.fp4_gemm_experts(off, hc, hs, *self.w2[:2], dtype=torch.bfloat16)
        y = mx.fp4_expert_combine(z, rows, weights, residual=res)
        dz, dw = mx.fp4_expert_combine_backward(dy, z, slots, rows, weights)
        dzr, dzs, dzc, dzcs = mx.fp4_quantize_dual(dz, mx.FP4_SR, 7, 1, 32, mask)
        dh = mx.fp4_gemm_experts(off, dzr, dzs, *self.w2[2:])
        dw2 = mx.fp4_gemm_experts_wgrad(off, dzc, dzcs, htc, hts)
        (dar, das), (dbr, dbs), (dac, dacs), (dbc, dbcs) = mx.fp4_swiglu_backward_producer(dh, a, b, 7, 2, 3, mask)
        dxs = mx.fp4_gemm_experts(off, dar, das, *self.w1c, dtype=torch.bfloat16, pair=[dbr, dbs, *self.w3c])
        dw1 = mx.fp4_gemm_experts_wgrad(off, dac, dacs, *xt)
        dw3 = mx.fp4_gemm_experts_wgrad(off, dbc, dbcs, *xt)
        dx = mx.fp4_expert_combine(dxs, rows)
        return dict(off=off, slots=slots, rows=rows, xs=xs, xc=xc, xsc=xsc, a=a, b=b, hc=hc, hs=hs, htc=htc, hts=hts, z=z, y=y, dz=dz,
                    dw=dw, dzr=dzr, dzs=dzs, dzc=dzc, dzcs=dzcs, dh=dh, dw2=dw2, dxs=dxs, dw1=dw1, dw3=dw3, dx=dx, dar=dar, das=das,
                    dbr=dbr, dbs=dbs, dac=dac, dacs=dacs, dbc=dbc, dbcs=dbcs, xtc=xt[0], xts=xt[1])


def inputs(layer, t, k, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(layer.E)[:k] for _ in range(t)]).astype(np.int32)
    ids[-1] = -1
    w = rng.random((t, k)).astype(np.float32)
    return (bf16(synthetic.tensor((t, layer.D), seed=seed)), dev(ids), dev(w), bf16(synthetic.tensor((t, layer.D), seed=seed + 1)),
            bf16(synthetic.tensor((t, layer.D), std=1e-2, seed=seed + 2)))


@pytest.mark.parametrize("E,D,Fh,t,k", [(5, 96, 64, 70, 2), (3, 256, 288, 300, 2)])
def test_training_step(gpu_lib, E, D, Fh, t, k):
    """Each call of the step against float64 on that call's own inputs."""
    layer = Layer(gpu_lib, E, D, Fh)
    x, ids, w, res, dy = inputs(layer, t, k, 3)
    r = layer.step(x, ids, w, res, dy)
    off, slots, rows = (host(r[n]) for n in ("off", "slots", "rows"))
    assert all(np.array_equal(g, v) for g, v in zip((off, slots, rows), X.sort(host(ids), E, 32)))
    assert np.array_equal(bits(r["xs"]), X.gather(bits(x), slots, k))
    wc, ws = Q.quantize_rows(bits(r["xs"]))
    assert np.array_equal(host(r["xc"]), wc) and np.array_equal(host(r["xsc"]), ws)

    def dec(c, s):
        return F.decode(host(r[c]), host(r[s]))

    def seg(e):
        return slice(off[e], off[e + 1])

    def weights(ws, e):
        return F.decode(host(ws[0][e]), host(ws[1][e]))

    xd, hd, dzd, dad, dbd = dec("xc", "xsc"), dec("hc", "hs"), dec("dzr", "dzs"), dec("dar", "das"), dec("dbr", "dbs")
    a64, z64, dh64, dxs64 = (np.zeros(host(r[n]).shape) for n in ("a", "z", "dh", "dxs"))
    for e in range(E):
        a64[seg(e)] = xd[seg(e)] @ weights(layer.w13, e)[:Fh].T
        z64[seg(e)] = hd[seg(e)] @ weights(layer.w2, e).T
        dh64[seg(e)] = dzd[seg(e)] @ weights(layer.w2[2:], e).T
        dxs64[seg(e)] = dad[seg(e)] @ weights(layer.w1c, e).T + dbd[seg(e)] @ weights(layer.w3c, e).T
        for name, left, right in (("dw2", ("dzc", "dzcs"), ("htc", "hts")), ("dw1", ("dac", "dacs"), ("xtc", "xts")),
                                  ("dw3", ("dbc", "dbcs"), ("xtc", "xts"))):
            assert close(host(r[name])[e], dec(*left)[:, seg(e)] @ dec(*right)[:, seg(e)].T, 1e-5), name
    for name, want, tol in (("a", a64, H), ("z", z64, H), ("dh", dh64, 1e-5), ("dxs", dxs64, H)):
        assert close(host(r[name]), want, tol), name
        assert (host(r[name])[slots < 0] == 0).all(), name
    f = lambda n: host(r[n]).astype(np.float64)  # noqa: E731
    assert close(f("y"), X.combine(f("z"), rows, host(w), host(res).astype(np.float64))[0], H)
    dz64, dw64, _ = X.combine_backward(host(dy).astype(np.float64), f("z"), rows, host(w))
    assert close(f("dz"), dz64, H) and close(f("dw"), dw64, 1e-5)
    assert close(f("dx"), X.combine(f("dxs"), rows)[0], H)
    assert (host(r["dx"])[-1] == 0).all() and np.array_equal(host(r["y"])[-1], host(res)[-1])   # the unrouted token


def test_the_step_is_the_same_again_on_a_stream_and_in_a_graph(gpu_lib):
    layer = Layer(gpu_lib, 4, 256, 96)
    args = inputs(layer, 200, 2, 9)
    want = {n: host(v) for n, v in layer.step(*args).items()}

    def same(r):
        return all(np.array_equal(host(v), want[n], equal_nan=False) for n, v in r.items())

    assert same(layer.step(*args))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = layer.step(*args)
    torch.cuda.current_stream().wait_stream(s)
    assert same(r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = layer.step(*args)
    other = inputs(layer, 200, 2, 10)
    other_want = {n: host(v) for n, v in layer.step(*other).items()}
    saved = [v.clone() for v in args]
    for turn in range(3):
        for v in r.values():                               # what a replay does not write would show
            v.view(torch.uint8).fill_(0xFF if turn else 0x5A)
        graph.replay()
        assert same(r)
        assert all(np.array_equal(host(v), other_want[n]) for n, v in layer.step(*other).items())   # eager work between
        for v, o in zip(args, other):                      # and other inputs in the same buffers
            v.copy_(o)
        graph.replay()
        assert all(np.array_equal(host(v), other_want[n]) for n, v in r.items())
        for v, o in zip(args, saved):
            v.copy_(o)


def test_two_streams_at_once(gpu_lib):
    """The calls keep nothing between them: two layers' steps interleaved on two streams."""
    layers = [Layer(gpu_lib, 4, 96, 64), Layer(gpu_lib, 3, 256, 96)]
    args = [inputs(layers[0], 300, 2, 1), inputs(layers[1], 150, 3, 2)]
    want = [{n: host(v) for n, v in la.step(*ar).items()} for la, ar in zip(layers, args)]
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        got = []
        for la, ar, s in zip(layers, args, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(la.step(*ar))
        for s in streams:
            s.synchronize()
        for g, w in zip(got, want):
            assert all(np.array_equal(host(v), w[n]) for n, v in g.items())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("t", [1, 5])
def test_decoded_tokens(gpu_lib, t, kind):
    """sort, gather, gated few-row product, product, combine for a few tokens, against float64."""
    mx, (E, D, Fh, k) = gpu_lib, (6, 288, 160, 2)
    layer = Layer(mx, E, D, Fh)
    rng = np.random.default_rng(t)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(t)])
    w = rng.random((t, k)).astype(np.float32)
    x, res = bf16(synthetic.tensor((t, D), seed=1)), bf16(synthetic.tensor((t, D), seed=2))
    off, slots, rows = mx.fp4_expert_sort(dev(ids), E, 1)
    xs, codes, scales = mx.fp4_expert_gather(x, slots, k, fmt=mx.FP4_E4M3)
    args = (xs, None) if kind == "bf16" else (codes, scales)
    h = mx.fp4_swiglu_matvec_experts(off, args[0], *layer.w13[:2], x_scales=args[1])
    z = mx.fp4_matvec_experts(off, h, *layer.w2[:2])
    y = host(mx.fp4_expert_combine(z, rows, dev(w), residual=res))
    want = host(res).astype(np.float64)
    for i in range(t):
        for j in range(k):
            e = ids[i, j]
            w13, w2 = (F.decode(host(m[0][e]), host(m[1][e])) for m in (layer.w13, layer.w2))
            ab = w13 @ host(x)[i].astype(np.float64)
            want[i] += w[i, j] * (w2 @ (A.value(ab[:Fh], A.SILU) * ab[Fh:]))
    # a, b, h and y each rounded to bf16; the E4M3 codes of x carry four bits
    assert close(y, want, 4 * H if kind == "bf16" else 2.0 ** -4)


def test_ungated_ffn_and_its_gradients(gpu_lib):
    """y = gelu(x W1^T + b1) W2^T + b2 + x and the gradients of that, call by call
    against float64; the bias' and the input's gradients also by differences."""
    mx, (t, D, Fh) = gpu_lib, (96, 288, 256)
    w1 = [dev(v) for v in Q.quantize_w2d32(synthetic.tensor((Fh, D), std=0.06, seed=1), 0.87)]
    w2 = [dev(v) for v in Q.quantize_w2d32(synthetic.tensor((D, Fh), std=0.06, seed=2), 0.87)]
    b1, b2 = torch.randn(Fh, device="cuda"), torch.randn(D, device="cuda").bfloat16()
    x = bf16(synthetic.tensor((t, D), seed=3))
    xq = mx.fp4_quantize_rows(x)
    h, z = mx.fp4_gemm_act(*xq, *w1[:2], mx.FP4_ACT_GELU, bias=b1, emit_z=True)
    hq = mx.fp4_quantize_rows(h)
    y, _ = mx.fp4_gemm_act(*hq, *w2[:2], bias=b2, residual=x, dtype=torch.float32)
    X64, H64, W1, W2 = (F.decode(host(a), host(b)) for a, b in (xq, hq, w1[:2], w2[:2]))
    z64 = X64 @ W1.T + host(b1)
    assert close(host(z), z64, H) and close(host(h), A.value(z64, A.GELU), H)
    assert close(host(y), H64 @ W2.T + host(b2) + host(x), 1e-5)
    # L = <dy, f(z) W2^T>: the gradients of z and of the bias
    dy = synthetic.tensor((t, D), std=1e-2, seed=4)
    dyq = mx.fp4_quantize_rows(bf16(dy))
    dh = mx.fp4_gemm(*dyq, *w2[2:])
    dz, db1 = mx.fp4_act_backward(dh, z, mx.FP4_ACT_GELU)
    slope = A.slope(host(z), A.GELU)
    assert close(host(dz), host(dh) * slope, H) and close(host(db1), (host(dh) * slope).sum(0), 1e-5)
    zz, dh64, step = host(z).astype(np.float64), host(dh).astype(np.float64), 1e-5
    loss = lambda zv: (dh64 * A.value(zv, A.GELU)).sum(0)  # noqa: E731
    diff = (loss(zz + step) - loss(zz - step)) / (2 * step)
    assert close(host(db1), diff, 1e-5)
    dx = mx.fp4_gemm(*mx.fp4_quantize_dual(dz, mx.FP4_SR, 1, 1)[:2], *w1[2:])
    assert close(host(dx), host(dz).astype(np.float64) @ F.decode(host(w1[0]), host(w1[1])), 0.2)   # four-bit stochastic codes
    few = mx.fp4_matvec_act(x[:3], *w1[:2], mx.FP4_ACT_GELU, bias=b1)
    assert close(host(few), A.value(host(x)[:3].astype(np.float64) @ W1.T + host(b1), A.GELU), H)


def test_tensors_that_do_not_fit_are_refused(gpu_lib):
    mx = gpu_lib
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    g = (u8(4, 32), u8(4, 2), u8(32, 32), u8(32, 2))       # m = 4, n = 32, k = 64
    bad = [lambda: mx.fp4_gemm_act(g[0], u8(4, 3), *g[2:]), lambda: mx.fp4_gemm_act(*g[:2], u8(32, 48), u8(32, 3)),
           lambda: mx.fp4_gemm_act(*g, bias=f32(31)), lambda: mx.fp4_gemm_act(*g, bias=i32(32)), lambda: mx.fp4_gemm_act(*g, residual=b16(4, 31)),
           lambda: mx.fp4_gemm_act(*g, residual=f32(4, 32)), lambda: mx.fp4_gemm_act(*g, dtype=torch.float16), lambda: mx.fp4_gemm_act(*g, 7),
           lambda: mx.fp4_gemm_act(*g, y=f32(4, 33)), lambda: mx.fp4_gemm_act(*g, emit_z=True, z=b16(4, 31)), lambda: mx.fp4_gemm_act(g[0].t(), *g[1:]),
           lambda: mx.fp4_gemm_act(g[0].cpu(), *g[1:]),
           lambda: mx.fp4_matvec_act(b16(65, 64), g[2], g[3]), lambda: mx.fp4_matvec_act(b16(2, 32), g[2], g[3]),
           lambda: mx.fp4_matvec_act(b16(2, 64), g[2], g[3], residual=b16(3, 32)),
           lambda: mx.fp4_act_backward(f32(4, 32), b16(4, 64), 1), lambda: mx.fp4_act_backward(f32(4, 48), b16(4, 48), 1),
           lambda: mx.fp4_act_backward(f32(4, 32), b16(4, 32), 1, accumulate=True), lambda: mx.fp4_act_backward(f32(4, 32), f32(4, 32), 1),
           lambda: mx.fp4_expert_sort(i32(4), 3), lambda: mx.fp4_expert_sort(f32(4, 2), 3), lambda: mx.fp4_expert_sort(i32(4, 2), 0),
           lambda: mx.fp4_expert_sort(i32(4, 2), 1025), lambda: mx.fp4_expert_sort(i32(4, 2), 3, 16), lambda: mx.fp4_expert_sort(i32(2, 4).t(), 3),
           lambda: mx.fp4_expert_sort(i32(4, 2), 3, 32, out=(i32(4), i32(100), i32(4, 2))), lambda: mx.fp4_expert_capacity(4, 2, 3, 48 + 1),
           lambda: mx.fp4_expert_gather(b16(4, 48), i32(8), 2), lambda: mx.fp4_expert_gather(b16(4, 64), i32(8, 1), 2),
           lambda: mx.fp4_expert_gather(b16(4, 64), i32(8).long(), 2), lambda: mx.fp4_expert_gather(b16(4, 64), i32(8), 0),
           lambda: mx.fp4_expert_gather(f32(4, 64), i32(8), 2), lambda: mx.fp4_expert_gather(b16(4, 64), i32(8), 2, fmt=3),
           lambda: mx.fp4_expert_combine(f32(8, 64), i32(8)), lambda: mx.fp4_expert_combine(f32(8, 64), i32(4, 2), f32(4, 3)),
           lambda: mx.fp4_expert_combine(f32(8, 48), i32(4, 2)), lambda: mx.fp4_expert_combine(f32(8, 64), i32(4, 2), residual=b16(3, 64)),
           lambda: mx.fp4_expert_combine_backward(b16(4, 64), f32(8, 64), i32(7), i32(4, 2), f32(4, 2)),
           lambda: mx.fp4_expert_combine_backward(b16(3, 64), f32(8, 64), i32(8), i32(4, 2), f32(4, 2)),
           lambda: mx.fp4_expert_combine_backward(b16(4, 64), f32(8, 64), i32(8), i32(4, 2), None),
           lambda: mx.fp4_gemm_experts(i32(4), g[0], g[1], u8(2, 32, 32), u8(2, 32, 2)), lambda: mx.fp4_gemm_experts(i32(3), g[0], g[1], g[2], g[3]),
           lambda: mx.fp4_gemm_experts(i32(3), g[0], g[1], u8(2, 32, 16), u8(2, 32, 1)),
           lambda: mx.fp4_gemm_experts(i32(3), g[0], g[1], u8(2, 32, 32), u8(2, 32, 2), pair=[u8(5, 32), u8(5, 2), u8(2, 32, 32), u8(2, 32, 2)]),
           lambda: mx.fp4_gemm_experts(i32(3), g[0], g[1], u8(2, 32, 32), u8(2, 32, 2), dtype=torch.int32),
           lambda: mx.fp4_gemm_experts_wgrad(i32(3), *g), lambda: mx.fp4_gemm_experts_wgrad(i32(1), u8(32, 128), u8(32, 8), u8(32, 128), u8(32, 8)),
           lambda: mx.fp4_gemm_experts_wgrad(i32(3), u8(32, 128), u8(32, 8), u8(32, 128), u8(32, 8), accumulate=True),
           lambda: mx.fp4_gemm_experts_wgrad(i32(3), u8(32, 128), u8(32, 8), u8(32, 128), u8(32, 8), c=b16(2, 32, 32), accumulate=True),
           lambda: mx.fp4_swiglu_producer_experts(i32(3), u8(32, 32), u8(32, 2), u8(2, 33, 32), u8(2, 33, 2)),
           lambda: mx.fp4_swiglu_producer_experts(i32(3), u8(40, 32), u8(40, 2), u8(2, 64, 32), u8(2, 64, 2)),
           lambda: mx.fp4_matvec_experts(i32(3), b16(4, 32), u8(2, 32, 32), u8(2, 32, 2)),
           lambda: mx.fp4_matvec_experts(i32(3), u8(4, 64), u8(2, 32, 32), u8(2, 32, 2), x_scales=u8(4, 3)),
           lambda: mx.fp4_swiglu_matvec_experts(i32(3), b16(4, 64), u8(2, 33, 32), u8(2, 33, 2))]
    for i, call in enumerate(bad):
        with pytest.raises(mx.Fp4Error):
            call()
            pytest.fail(f"call {i} was not refused")
