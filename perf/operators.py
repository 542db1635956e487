"""The operators around the MXFP4 linear layer, as they are measured.

Five operators, each in a plain form of elementary torch operations and as the
package's own call:

  norm          s = bf16(dropout(x) + residual), rstd = 1/sqrt(mean(s^2) + eps),
                y = bf16(s rstd gamma), and y in E4M3 with one upward E8M0 scale
                per 32 values
  norm_grad     the gradients of that boundary: of the sum, of x and of gamma
  dropout       bf16(x keep 65536/(65536 - thr) [+ residual]), keep from a counter
  matvec        C = X dec(W)^T for a few rows of X, W in MXFP4 or NVFP4
  swiglu_matvec h = bf16(SiLU(a) b), a = bf16(X W1^T), b = bf16(X W3^T), few rows

A dropout draw is half of a Philox4x32-10 word: element c of row r has index
i = r * 8 ceil(cols / 8) + c and takes half i & 1 of word (i >> 1) & 3 of the
block at counter (lo32(i >> 3), hi32(i >> 3), lo32(offset), hi32(offset)) under
key (lo32(seed), hi32(seed)); it is kept iff the half is >= thr, where
thr = floor(65536 p + 1/2).
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-5
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token enters a layer: the sum and the norm, read by an 8-bit matvec next
        {"name": "norm_1x4096", "op": "norm", "t": 1, "d": 4096, "x": "bf16", "residual": True, "p": 0.0},
        # a training step of the 4096-wide layer: the product's fp32 output, dropout, residual
        {"name": "norm_8192x4096_dropout", "op": "norm", "t": 8192, "d": 4096, "x": "fp32", "residual": True, "p": 0.1},
        # a ragged batch of a narrow odd model width, the first norm of a stack (no residual)
        {"name": "norm_1001x1056", "op": "norm", "t": 1001, "d": 1056, "x": "bf16", "residual": False, "p": 0.0},
        # the same training step backwards: dY is the data gradient's fp32 output
        {"name": "norm_grad_8192x4096_dropout", "op": "norm_grad", "t": 8192, "d": 4096, "dy": "fp32", "ds": True, "p": 0.1},
        # a short ragged batch of the 8192-wide layer
        {"name": "norm_grad_515x8192", "op": "norm_grad", "t": 515, "d": 8192, "dy": "bf16", "ds": False, "p": 0.0},
        # dropout of the gated hidden activations
        {"name": "dropout_8192x14336", "op": "dropout", "rows": 8192, "cols": 14336, "x": "bf16", "residual": False, "p": 0.1},
        # a small odd-sized tensor of fp32 products added to the residual stream
        {"name": "dropout_127x4099_add", "op": "dropout", "rows": 127, "cols": 4099, "x": "fp32", "residual": True, "p": 0.25},
        # one token through the 4096 x 4096 attention projection
        {"name": "matvec_1_4096x4096", "op": "matvec", "m": 1, "n": 4096, "k": 4096, "x": "bf16", "w": "mxfp4"},
        # five drafted tokens through the stacked gate/up weights of the large FFN, from the norm's 8-bit output
        {"name": "matvec_5_57344x8192_e4m3", "op": "matvec", "m": 5, "n": 57344, "k": 8192, "x": "e4m3", "w": "mxfp4"},
        # a batch of 33 sequences through the down projection held in NVFP4
        {"name": "matvec_33_4096x14336_nv", "op": "matvec", "m": 33, "n": 4096, "k": 14336, "x": "bf16", "w": "nvfp4"},
        # one token through the gate/up half of the 14336-wide FFN
        {"name": "swiglu_matvec_1_14336x4096", "op": "swiglu_matvec", "m": 1, "f": 14336, "d": 4096, "x": "e4m3"},
        # a batch of 16 sequences through the same
        {"name": "swiglu_matvec_16_14336x4096", "op": "swiglu_matvec", "m": 16, "f": 14336, "d": 4096, "x": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "dropout", "matvec", "swiglu_matvec"))
    if op in ("norm", "norm_grad"):
        c = {"op": op, "t": _log(rng, 1, 8192), "d": 32 * _log(rng, 1, 256), "p": rng.choice((0.0, 0.1))}
        if op == "norm":
            return c | {"x": rng.choice(("bf16", "fp32")), "residual": rng.random() < 0.7}
        return c | {"dy": rng.choice(("bf16", "fp32")), "ds": rng.random() < 0.7}
    if op == "dropout":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 1, 14336), "x": rng.choice(("bf16", "fp32")),
                "residual": rng.random() < 0.5, "p": rng.choice((0.1, 0.25, 0.5))}
    m = _log(rng, 1, 64)
    if op == "matvec":
        w = rng.choice(("mxfp4", "mxfp4", "nvfp4"))
        return {"op": op, "m": m, "n": _log(rng, 1, 28672), "k": 32 * _log(rng, 1, 448), "w": w,
                "x": "bf16" if w == "nvfp4" else rng.choice(("bf16", "e4m3"))}
    return {"op": op, "m": m, "f": _log(rng, 1, 14336), "d": 32 * _log(rng, 1, 256), "x": rng.choice(("bf16", "e4m3"))}


# ------------------------------------------------------------------ inputs


def _activations(g, *shape):
    """N(0, 1) with one entry in a thousand twenty times as large."""
    x = torch.randn(shape, device="cuda", generator=g)
    return torch.where(torch.rand(shape, device="cuda", generator=g) < 1e-3, 20 * x, x)


def _pow2(e):
    """2^e in fp32 from its bits, -126 <= e <= 127 (a power function may be a rounding off)."""
    return ((e + 127).int() << 23).view(torch.float32)


def _upward(amax, q_max):
    """The smallest e with amax <= q_max 2^e, at least -127 (q_max = f 2^E, f in [1/2, 1))."""
    f, big = math.frexp(q_max)
    mant, ex = torch.frexp(amax)
    e = ex - big + (mant > f)
    return torch.where(amax > 0, e, -127).clamp(min=-127)


def _e4m3(y):
    """(codes, scales) of fp32 rows: E4M3 values in blocks of 32 under upward E8M0 scales."""
    b = y.unflatten(-1, (-1, 32))
    e = _upward(b.abs().amax(-1), 448.0)
    codes = (b * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _nibbles(v):
    """E2M1 codes of values already divided by their scales, two per byte."""
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda")
    code = torch.bucketize(v.abs(), mids, out_int32=True) + 8 * (v < 0)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def _weights(g, n, k, kind):
    """N(0, 0.02) weights as codes and group scales, row-major along k."""
    w = 0.02 * torch.randn((n, k), device="cuda", generator=g)
    if kind == "mxfp4":
        b = w.unflatten(-1, (-1, 32))
        e = _upward(b.abs().amax(-1), 6.0)
        return {"codes": _nibbles((b * _pow2(-e)[..., None]).flatten(-2)), "scales": (e + 127).to(torch.uint8)}
    b = w.unflatten(-1, (-1, 16))
    factor = w.abs().amax() / 2688
    d = (b.abs().amax(-1) / (6 * factor)).to(torch.float8_e4m3fn)
    return {"codes": _nibbles((b / (d.float() * factor)[..., None]).flatten(-2)), "scales": d.view(torch.uint8),
            "factor": factor.reshape(1)}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 17)
    op, s = case["op"], {"case": case, "seed": 0x1234_5678_0000 + seed, "offset": 3 * seed + 1}
    kind = lambda x, name: x if name == "fp32" else x.bfloat16()  # noqa: E731
    if op == "norm":
        t, d = case["t"], case["d"]
        s["x"] = kind(_activations(g, t, d), case["x"])
        s["residual"] = _activations(g, t, d).bfloat16() if case["residual"] else None
        s["gamma"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    elif op == "norm_grad":
        t, d = case["t"], case["d"]
        s["dy"] = kind(1e-3 * torch.randn((t, d), device="cuda", generator=g), case["dy"])
        s["s"] = _activations(g, t, d).bfloat16()
        s["rstd"] = 1 / (s["s"].float().square().mean(-1) + EPS).sqrt()
        s["gamma"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
        s["ds"] = (1e-3 * torch.randn((t, d), device="cuda", generator=g)).bfloat16() if case["ds"] else None
    elif op == "dropout":
        r, c = case["rows"], case["cols"]
        # rows are kept at a pitch of a multiple of eight elements
        rows = lambda x: torch.nn.functional.pad(x, (0, -c % 8))[:, :c]  # noqa: E731
        s["x"] = rows(kind(_activations(g, r, c), case["x"]))
        s["residual"] = rows(_activations(g, r, c).bfloat16()) if case["residual"] else None
    else:
        n, k = (case["n"], case["k"]) if op == "matvec" else (2 * case["f"], case["d"])
        s["w"] = _weights(g, n, k, case.get("w", "mxfp4"))
        x = _activations(g, case["m"], k)
        if case["x"] == "e4m3":
            codes, scales = _e4m3(x)
            s["x"], s["x_scales"] = codes.view(torch.uint8), scales.view(torch.uint8)
        else:
            s["x"], s["x_scales"] = x.bfloat16(), None
    return s


def work(case):
    op, size = case["op"], {"bf16": 2, "fp32": 4, "e4m3": 1}
    if op == "norm":
        n = case["t"] * case["d"]
        return {"bytes": n * (size[case["x"]] + 2 * case["residual"] + 2 + 1 + 1 / 32) + 4 * case["t"] + 2 * case["d"],
                "flops": 6 * n}
    if op == "norm_grad":
        n = case["t"] * case["d"]
        return {"bytes": n * (size[case["dy"]] + 2 + 2 * case["ds"] + 2 + 2 * (case["p"] > 0)) + 4 * case["t"] + 6 * case["d"],
                "flops": 12 * n}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + 2 * case["residual"] + 2), "flops": 2 * n}
    m, n, k = (case["m"], case["n"], case["k"]) if op == "matvec" else (case["m"], 2 * case["f"], case["d"])
    x = m * k * (2 if case["x"] == "bf16" else 1 + 1 / 32)
    w = n * k * (0.5 + (1 / 32 if case.get("w", "mxfp4") == "mxfp4" else 1 / 16))
    return {"bytes": x + w + (4 * m * n if op == "matvec" else m * n), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ plain forms


def _keep(rows, cols, p, seed, offset):
    """(kept elements, scale of the kept ones): Philox4x32-10 in 64-bit integers (products wrap modulo 2^64)."""
    thr = math.floor(65536 * p + 0.5)
    low = 0xFFFFFFFF
    per = -(-cols // 8)
    i = torch.arange(rows * per, device="cuda")
    x, y = i & low, i >> 32
    z, w = torch.full_like(i, offset & low), torch.full_like(i, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = x * 0xD2511F53, z * 0xCD9E8D57
        x, y, z, w = ((b >> 32) & low) ^ y ^ k0, b & low, ((a >> 32) & low) ^ w ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((x, y, z, w), -1)
    halves = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(rows, 8 * per)[:, :cols]
    return halves >= thr, (65536 / (65536 - thr) if thr < 65536 else 0.0)


def _decoded(codes, scales, group):
    """fp32 values of E2M1 codes under one fp32 scale per `group` values."""
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda")
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, group)) * scales[..., None]).flatten(-2)


def _e8m0(scales):
    return scales.view(torch.float8_e8m0fnu).float()


def _product(st):
    w, x = st["w"], st["x"]
    if st["x_scales"] is not None:
        x = (x.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * _e8m0(st["x_scales"])[..., None]).flatten(-2)
    if "factor" in w:
        return w["factor"] * (x.float() @ _decoded(w["codes"], w["scales"].view(torch.float8_e4m3fn).float(), 16).t())
    return x.float() @ _decoded(w["codes"], _e8m0(w["scales"]), 32).t()


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        v = st["x"].float()
        if case["p"] > 0:
            keep, scale = _keep(*v.shape, case["p"], st["seed"], st["offset"])
            v = torch.where(keep, v * scale, 0.0)
        s = (v if st["residual"] is None else v + st["residual"].float()).bfloat16()
        v = s.float()
        rstd = 1 / (v.square().mean(-1) + EPS).sqrt()
        y = (v * rstd[:, None] * st["gamma"].float()).bfloat16()
        return {"sum": s, "rstd": rstd, **dict(zip(("codes", "scales"), _e4m3(y.float())))}
    if op == "norm_grad":
        dy, r = st["dy"].float(), st["rstd"][:, None]
        xhat, g = st["s"].float() * r, dy * st["gamma"].float()
        ds = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if st["ds"] is not None:
            ds = ds + st["ds"].float()
        out = {"dsum": ds.bfloat16(), "dgamma": (dy * xhat).sum(0)}
        if case["p"] > 0:
            keep, scale = _keep(*ds.shape, case["p"], st["seed"], st["offset"])
            out["dx"] = torch.where(keep, ds * scale, 0.0).bfloat16()
        return out
    if op == "dropout":
        keep, scale = _keep(*st["x"].shape, case["p"], st["seed"], st["offset"])
        v = torch.where(keep, st["x"].float() * scale, 0.0)
        return (v if st["residual"] is None else v + st["residual"].float()).bfloat16()
    if op == "matvec":
        return _product(st)
    a, b = _product(st).bfloat16().float().chunk(2, -1)
    return (a / (1 + torch.exp(-a)) * b).bfloat16()


# ------------------------------------------------------------------ the package's calls


_package = None


def _own(st):
    global _package
    if _package is None:
        import precision_mxfp4_producers_amd
        _package = precision_mxfp4_producers_amd
    mx, case = _package, st["case"]
    op = case["op"]
    if op == "norm":
        s, rstd, _, codes, scales = mx.fp4_rmsnorm_producer(st["x"], st["gamma"], EPS, residual=st["residual"], p=case["p"],
                                                            seed=st["seed"], offset=st["offset"], fmt=mx.FP4_E4M3)
        return {"sum": s, "rstd": rstd, "codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
    if op == "norm_grad":
        dsum, dx, dgamma = mx.fp4_rmsnorm_backward(st["dy"], st["s"], st["rstd"], st["gamma"], ds=st["ds"], p=case["p"],
                                                   seed=st["seed"], offset=st["offset"])
        return {"dsum": dsum, "dgamma": dgamma} | ({"dx": dx} if case["p"] > 0 else {})
    if op == "dropout":
        return mx.fp4_dropout(st["x"], case["p"], st["seed"], st["offset"], residual=st["residual"])
    w = st["w"]
    if op == "matvec":
        if "factor" in w:
            return mx.fp4_nv_matvec(st["x"], w["codes"], w["scales"], w["factor"])
        return mx.fp4_matvec(st["x"], w["codes"], w["scales"], x_scales=st["x_scales"])
    return mx.fp4_swiglu_matvec(st["x"], w["codes"], w["scales"], x_scales=st["x_scales"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64-bit values


def _drawn(rows, cols, p, seed, offset):
    """The kept elements and their scale, from numpy's unsigned arithmetic on 32-bit lanes."""
    thr, per = int(np.floor(np.float64(p) * 65536 + 0.5)), (cols + 7) // 8
    u = np.uint64
    m32, sh = u(0xFFFFFFFF), u(32)
    block = np.arange(rows * per, dtype=u)
    c = [block & m32, block >> sh, np.full(rows * per, offset & 0xFFFFFFFF, u), np.full(rows * per, offset >> 32, u)]
    for r in range(10):
        key = [u((seed + r * 0x9E3779B9) & 0xFFFFFFFF), u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)]
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> sh) ^ c[1] ^ key[0], p1 & m32, (p0 >> sh) ^ c[3] ^ key[1], p0 & m32]
    keep = np.empty((rows * per, 8), bool)
    for j in range(4):
        keep[:, 2 * j] = (c[j] & u(0xFFFF)) >= u(thr)
        keep[:, 2 * j + 1] = (c[j] >> u(16)) >= u(thr)
    keep = torch.from_numpy(keep.reshape(rows, 8 * per)[:, :cols].copy()).cuda()
    return keep, (1.0 / (1.0 - thr / 65536.0) if thr < 65536 else 0.0)


def _unit(e):
    """2^e in float64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rounded(v):
    """float64 values rounded once to bf16 (nearest, ties to even), as float64; normal range."""
    unit = _unit(torch.frexp(v).exponent - 8)
    return torch.round(v / unit) * unit


def _fp4_value(nibble):
    """E2M1 by its fields: exponent e, fraction f, sign."""
    e, f, sign = (nibble >> 1) & 3, nibble & 1, 1.0 - 2.0 * (nibble >> 3).double()
    mag = torch.where(e > 0, (1 + f.double() / 2) * _unit(e.long() - 1), f.double() / 2)
    return sign * mag


def _e4m3_value(byte):
    b = byte.int()
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + f / 8) * _unit(e - 7), f / 512)
    return torch.where(b >= 128, -mag, mag)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad", "dropout"):
        shape = (case["rows"], case["cols"]) if op == "dropout" else (case["t"], case["d"])
        keep, scale = _drawn(*shape, case["p"], st["seed"], st["offset"])
    if op == "dropout":
        v = st["x"].double().mul(scale).masked_fill(~keep, 0.0)
        return v if st["residual"] is None else v + st["residual"].double()
    if op == "norm":
        v = st["x"].double().mul(scale).masked_fill(~keep, 0.0)
        s = _rounded(v if st["residual"] is None else v + st["residual"].double())
        rstd = torch.rsqrt((s * s).sum(-1) / case["d"] + EPS)
        y = _rounded(s * rstd.unsqueeze(-1) * st["gamma"].double()).reshape(case["t"], -1, 32)
        top = y.abs().max(-1).values
        # the smallest e with 448 2^e >= top: the exponent of top / 448, or one below where that is a power of two
        e = torch.frexp(top / 448).exponent
        e = torch.where(448 * _unit(e - 1) >= top, e - 1, e).clamp(min=-127)
        q = y / _unit(e).unsqueeze(-1)
        step = _unit(torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent - 4)
        q = (torch.round(q / step) * step).reshape(case["t"], case["d"])
        return {"sum": s, "rstd": rstd, "codes": q, "scales": _unit(e)}
    if op == "norm_grad":
        dy, s, r = st["dy"].double(), st["s"].double(), st["rstd"].double().unsqueeze(-1)
        g = dy * st["gamma"].double()
        ds = r * g - s * r.pow(3) * (g * s).sum(-1, keepdim=True) / case["d"]
        if st["ds"] is not None:
            ds += st["ds"].double()
        out = {"dsum": ds, "dgamma": (dy * s * r).sum(0)}
        return out | ({"dx": ds.mul(scale).masked_fill(~keep, 0.0)} if case["p"] > 0 else {})
    codes, scales = st["w"]["codes"], st["w"]["scales"]
    if "factor" in st["w"]:
        delta, group = _e4m3_value(scales) * st["w"]["factor"].double(), 16
    else:
        delta, group = _unit(scales.long() - 127), 32
    x = st["x"].double()
    if st["x_scales"] is not None:
        x = _e4m3_value(st["x"]) * _unit(st["x_scales"].long() - 127).repeat_interleave(32, -1)
    out = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float64, device="cuda")
    for at in range(0, codes.shape[0], 4096):  # rows of W in parts: the 64-bit values take sixteen times the codes' room
        part = codes[at:at + 4096]
        w = torch.empty((part.shape[0], 2 * part.shape[1]), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = _fp4_value(part & 15), _fp4_value(part >> 4)
        w *= delta[at:at + 4096].repeat_interleave(group, -1)
        out[:, at:at + 4096] = x @ w.t()
    if op == "matvec":
        return out
    a, b = _rounded(out[:, :case["f"]]), _rounded(out[:, case["f"]:])
    return a * torch.sigmoid(a) * b
