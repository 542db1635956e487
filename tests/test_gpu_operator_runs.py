"""The norm, dropout and few-row products as they are used: a training block
forwards and backwards, a decoded token's FFN, replayed graphs and other
streams.  Every step is checked against the oracle on its actual inputs."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N
from oracle import quant as Q

pytestmark = pytest.mark.gpu
H, U = 2.0 ** -8, 2.0 ** -24


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def bits(t):
    return host(t.contiguous().view(torch.int16)).view(np.uint16)


def val(t):
    return F.bf16_bits_to_f64(bits(t))


def make(t, d, f, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0: (k * torch.randn(s, device="cuda", generator=g))  # noqa: E731
    return {"x": r(t, d), "res": r(t, d).bfloat16(), "gamma": (1 + 0.1 * r(d)).bfloat16(),
            "w1": r(f, d, k=0.05).bfloat16(), "w3": r(f, d, k=0.05).bfloat16(), "w2": r(d, f, k=0.05).bfloat16(),
            "dy": r(t, d, k=1e-3).bfloat16()}


def train_step(mx, v, p, seed, mask):
    """Pre-norm gated FFN block with dropout on the incoming branch and on the
    block's output, and its backward pass to the block's inputs."""
    w1, w3, w2 = (mx.fp4_quantize_w2d32(v[k], 0.87) for k in ("w1", "w3", "w2"))
    s, rstd, y, yc, ys = mx.fp4_rmsnorm_producer(v["x"], v["gamma"], 1e-5, v["res"], p, seed, 1, mx.FP4_E2M1, emit_y=True)
    w13 = (torch.cat([w1[0], w3[0]]), torch.cat([w1[1], w3[1]]))
    a, b, hc, hs, htc, hts = mx.fp4_swiglu_producer(yc, ys, *w13, mask)
    out32 = mx.fp4_gemm(hc, hs, w2[0], w2[1])
    out = mx.fp4_dropout(out32, p, seed, 2, residual=s)
    # backwards: the output's gradient reaches s directly and through the FFN
    dout = mx.fp4_dropout(v["dy"], p, seed, 2)
    dr = mx.fp4_quantize_rows(dout, mx.FP4_SR, seed, 3)
    dh = mx.fp4_gemm(dr[0], dr[1], w2[2], w2[3])
    da, db, dac, dbc = mx.fp4_swiglu_backward_producer(dh, a, b, seed, 4, 5, mask)
    dyn = mx.fp4_gemm_pair(*da, w1[2], w1[3], *db, w3[2], w3[3])
    dsum, dx, dgamma = mx.fp4_rmsnorm_backward(dyn, s, rstd, v["gamma"], ds=v["dy"], p=p, seed=seed, offset=1)
    return dict(s=s, rstd=rstd, y=y, yc=yc, ys=ys, hc=hc, hs=hs, out32=out32, out=out, dout=dout, dyn=dyn, dsum=dsum,
                dx=dx, dgamma=dgamma)


def test_training_block(gpu_lib):
    mx, p, seed = gpu_lib, 0.1, 42
    t, d, f = 160, 256, 352
    v = make(t, d, f, 1)
    o = train_step(mx, v, p, seed, mx.fp4_sign_mask_from_seed(0))
    sb = N.dropout_bits(host(v["x"]), p, seed, 1, bits(v["res"]))
    assert np.array_equal(bits(o["s"]), sb)
    codes, scales = Q.quantize_rows(bits(o["y"]))
    assert np.array_equal(host(o["yc"]), codes) and np.array_equal(host(o["ys"]), scales)
    assert np.array_equal(bits(o["out"]), N.dropout_bits(host(o["out32"]), p, seed, 2, sb))
    assert np.array_equal(bits(o["dout"]), N.dropout_bits(val(v["dy"]).astype(np.float32), p, seed, 2))
    r, s64, g64 = host(o["rstd"]).astype(np.float64), F.bf16_bits_to_f64(sb), val(v["gamma"])
    dyn, ds64 = host(o["dyn"]).astype(np.float64), val(v["dy"])
    want, wg = N.rmsnorm_backward(dyn, s64, r, g64, ds64)
    xh, g = s64 * r[:, None], dyn * g64
    size = r[:, None] * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True)) + np.abs(ds64)
    assert (np.abs(val(o["dsum"]) - want) <= H * np.abs(want) + 64 * U * size).all()
    keep, sc = N.keep_mask(t, d, p, seed, 1), float(N.keep_scale(p))
    assert (np.abs(val(o["dx"]) - np.where(keep, want * sc, 0)) <= H * sc * np.abs(want) + 64 * U * sc * size).all()
    assert (np.abs(host(o["dgamma"]) - wg) <= 65 * U * np.abs(dyn * xh).sum(axis=0)).all()


def decode_token(mx, v, w13, w2, x, res):
    s, rstd, _, c, sc = mx.fp4_rmsnorm_producer(x, v["gamma"], 1e-5, res)
    h = mx.fp4_swiglu_matvec(c, *w13, x_scales=sc)
    out = mx.fp4_matvec(h, w2[0], w2[1])
    s2 = mx.fp4_rmsnorm_producer(out, v["gamma"], 1e-5, s, emit_codes=False, emit_y=True)
    return s, c, sc, h, out, s2[0], s2[2]


@pytest.mark.parametrize("m", [1, 5, 33])
def test_decoded_tokens(gpu_lib, m):
    mx = gpu_lib
    d, f = 512, 736
    v = make(m, d, f, 2)
    w1, w3, w2 = (mx.fp4_quantize_w2d32(v[k], 0.87) for k in ("w1", "w3", "w2"))
    w13 = (torch.cat([w1[0], w3[0]]), torch.cat([w1[1], w3[1]]))
    s, c, sc, h, out, s2, y2 = decode_token(mx, v, w13, w2, v["x"], v["res"])
    x64 = N.decode_e4m3(host(c), host(sc))
    ab = x64 @ F.decode(host(w13[0]), host(w13[1])).T
    a, b = ab[:, :f], ab[:, f:]
    want = a / (1 + np.exp(-a)) * b
    # two rounded factors and the result: the relative error of the whole row in the 2-norm
    assert np.linalg.norm(val(h) - want) <= 3 * H * np.linalg.norm(want)
    h64, w64 = val(h), F.decode(host(w2[0]), host(w2[1]))
    assert G.within_bound(host(out), h64 @ w64.T, np.abs(h64) @ np.abs(w64).T).all()
    sb = N.dropout_bits(host(out), 0.0, 0, 0, bits(s))
    assert np.array_equal(bits(s2), sb)
    y64 = N.rmsnorm(F.bf16_bits_to_f64(sb), val(v["gamma"]), 1e-5)[1]
    assert (np.abs(val(y2) - y64) <= (H + 36 * U) * np.abs(y64)).all()


def run_all(mx, v, w, p, seed):
    """Every new call once; the outputs."""
    x, res, gamma = v["x"], v["res"], v["gamma"]
    s, rstd, y, c, sc = mx.fp4_rmsnorm_producer(x, gamma, 1e-5, res, p, seed, 1, emit_y=True)
    b = mx.fp4_rmsnorm_backward(x, s, rstd, gamma, res, p, seed, 1)
    dr = mx.fp4_dropout(x, p, seed, 2, res)
    h = mx.fp4_swiglu_matvec(c[:7], *w["w13"], x_scales=sc[:7])
    o = mx.fp4_matvec(h, *w["w2"])
    nv = mx.fp4_nv_matvec(h, *w["nv2"])
    return [s, rstd, y, c, sc, *b, dr, h, o, nv]


def prepared(mx, seed):
    v = make(96, 256, 320, seed)
    w1, w3, w2 = (mx.fp4_quantize_w2d32(v[k], 0.87) for k in ("w1", "w3", "w2"))
    nv = mx.fp4_nv_quantize_w2d16(v["w2"])
    return v, {"w13": (torch.cat([w1[0], w3[0]]), torch.cat([w1[1], w3[1]])), "w2": (w2[0], w2[1]),
               "nv2": (nv[0], nv[1], nv[4])}


def test_graphs_replayed_in_turn(gpu_lib):
    """Two captured graphs of every call, replayed several times in turn with
    eager work and new inputs between: each replay gives the eager bytes."""
    mx = gpu_lib
    sides = []
    for seed in (3, 4):
        v, w = prepared(mx, seed)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run_all(mx, v, w, 0.2, seed)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_all(mx, v, w, 0.2, seed)
        sides.append((seed, v, w, g, out))
    for turn in range(4):
        for seed, v, w, g, out in sides if turn % 2 else sides[::-1]:
            v["x"].copy_(torch.roll(v["x"], turn + 1, 0))
            g.replay()
            want = run_all(mx, v, w, 0.2, seed)
            torch.cuda.synchronize()
            for k, (a, b) in enumerate(zip(out, want)):
                assert torch.equal(a, b), (turn, seed, k)


def test_calls_on_two_streams(gpu_lib):
    """The same calls on two streams at once, with nothing shared but the inputs."""
    mx = gpu_lib
    v, w = prepared(mx, 5)
    want = run_all(mx, v, w, 0.1, 7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(run_all(mx, v, w, 0.1, 7))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_documented_usage(gpu_lib):
    """The documented usage, in small: a boundary with its backward pass and a decoded token."""
    mx, T, D = gpu_lib, 96, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (0.02 * torch.randn(D, D, device="cuda", generator=g)).bfloat16()
    wr, wrs, wc, wcs = mx.fp4_quantize_w2d32(w, 0.87)
    y = torch.randn(T, D, device="cuda", generator=g)
    dx = torch.randn(T, D, device="cuda", generator=g)
    gamma, res = torch.ones(D, device="cuda").bfloat16(), torch.zeros(T, D, device="cuda").bfloat16()
    s, rstd, yn, yc, ys = mx.fp4_rmsnorm_producer(y, gamma, 1e-5, residual=res, p=0.1, seed=7, offset=0, fmt=mx.FP4_E2M1,
                                                  emit_y=True)
    dres, dbranch, dgamma = mx.fp4_rmsnorm_backward(dx, s, rstd, gamma, p=0.1, seed=7, offset=0)
    assert dres.shape == dbranch.shape == (T, D) and dgamma.shape == (D,)
    out = mx.fp4_gemm(yc, ys, wr, wrs)
    ref, e = G.gemm_ref(host(yc), host(ys), host(wr), host(wrs))
    assert G.within_bound(host(out), ref, e).all()
    s1, r1, _, c8, s8 = mx.fp4_rmsnorm_producer(y[:1], gamma, residual=res[:1])
    one = mx.fp4_matvec(c8, wr, wrs, x_scales=s8)
    x64, w64 = N.decode_e4m3(host(c8), host(s8)), F.decode(host(wr), host(wrs))
    assert G.within_bound(host(one), x64 @ w64.T, np.abs(x64) @ np.abs(w64).T).all()
