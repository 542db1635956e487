"""Operators for layers of many experts and for products with an epilogue, as they are measured.

Three operators, each in a plain form of elementary torch operations and as the
package's own calls:

  tokens    tokens sorted by expert (offsets, slots, rows) with their
            activations gathered (dispatch), the experts' results weighted and
            added back (combine), and that sum's gradients (combine_grad)
  experts   C[r] = A[r] W_e^T for the rows of each expert's segment (rows),
            dW_e = A B_e^T over the segment's tokens (wgrad), both MXFP4, and
            bf16 or E4M3 activations of a few tokens against the 4-bit weights,
            plain or gated (few)
  act       z = A W^T + bias, y = act(z) + residual with MXFP4 operands (gemm),
            the same for a few rows of bf16 or E4M3 activations (few), and the
            gradients dz = dy act'(z), dbias = the column sums of dz (grad)

Order of the sorted tokens: slot t k + j holds token t's j-th expert; expert e
owns the rows offsets[e] .. offsets[e + 1] - 1, its slots in ascending order and
then padding up to a multiple of `align`; slots[r] is -1 and the row zero where
no token stands, rows[t][j] is -1 where ids[t][j] is no expert.  The buffers
hold capacity(t k, experts, align) rows.
"""

import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one decoded token enters a layer of eight experts, the 4096-wide model
        {"name": "dispatch_1x4096_e8k2", "op": "tokens", "form": "dispatch", "t": 1, "d": 4096, "e": 8, "k": 2,
         "align": 1, "codes": True},
        # a training step's tokens to 64 small experts, segments in whole blocks of 32 tokens
        {"name": "dispatch_8192x2048_e64k8", "op": "tokens", "form": "dispatch", "t": 8192, "d": 2048, "e": 64, "k": 8,
         "align": 32, "codes": False},
        # a batch of nine decoded tokens back onto the residual stream
        {"name": "combine_9x4096_e8k2", "op": "tokens", "form": "combine", "t": 9, "d": 4096, "e": 8, "k": 2, "align": 1,
         "z": "fp32", "residual": True},
        # the training step's experts' outputs back to their tokens
        {"name": "combine_8192x4096_e8k2", "op": "tokens", "form": "combine", "t": 8192, "d": 4096, "e": 8, "k": 2,
         "align": 32, "z": "bf16", "residual": True},
        # the same step backwards, 64 small experts
        {"name": "combine_grad_8192x2048_e64k8", "op": "tokens", "form": "combine_grad", "t": 8192, "d": 2048, "e": 64,
         "k": 8, "align": 32, "z": "bf16", "dy": "bf16"},
        # the gate and up products of 64 small experts, eight a token (training)
        {"name": "experts_8192_2048x2048_e64k8", "op": "experts", "form": "rows", "t": 8192, "n": 2048, "d": 2048, "e": 64,
         "k": 8, "out": "bf16"},
        # their weight gradients
        {"name": "experts_wgrad_8192_2048x2048_e64k8", "op": "experts", "form": "wgrad", "t": 8192, "n": 2048, "d": 2048,
         "e": 64, "k": 8},
        # one decoded token through the gate/up halves of its two 14336-wide experts
        {"name": "experts_few_1_14336x4096_e8k2", "op": "experts", "form": "few", "t": 1, "n": 14336, "d": 4096, "e": 8,
         "k": 2, "x": "bf16", "gate": True},
        # a decoding batch of 24 tokens through small experts' down projections
        {"name": "experts_few_24_2048x1056_e64k8", "op": "experts", "form": "few", "t": 24, "n": 2048, "d": 1056, "e": 64,
         "k": 8, "x": "e4m3", "gate": False},
        # the first product of an ungated FFN in training: bias, GELU, z kept for the backward pass
        {"name": "act_8192x14336x4096_gelu", "op": "act", "form": "gemm", "m": 8192, "n": 14336, "d": 4096, "act": "gelu",
         "bias": True, "residual": False, "out": "bf16", "z": True},
        # one token's down projection onto the residual stream
        {"name": "act_few_1_4096x14336", "op": "act", "form": "few", "m": 1, "n": 4096, "d": 14336, "act": "none",
         "bias": True, "residual": True, "out": "bf16", "x": "bf16"},
        # the training step backwards: dY is the data gradient's fp32 output
        {"name": "act_grad_8192x14336_gelu", "op": "act", "form": "grad", "m": 8192, "n": 14336, "act": "gelu", "dy": "fp32"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tokens", "tokens", "experts", "experts", "act"))
    if op == "act":
        form = rng.choice(("gemm", "few", "grad"))
        act = rng.choice(ACTS)
        if form == "grad":
            return {"op": op, "form": form, "m": _log(rng, 1, 8192), "n": 32 * _log(rng, 1, 448), "act": act,
                    "dy": rng.choice(("bf16", "fp32"))}
        c = {"op": op, "form": form, "m": _log(rng, 1, 64 if form == "few" else 8192), "n": 32 * _log(rng, 1, 448),
             "d": 32 * _log(rng, 1, 128), "act": act, "bias": rng.random() < 0.6, "residual": rng.random() < 0.5,
             "out": rng.choice(("bf16", "bf16", "fp32"))}
        return c | ({"x": rng.choice(("bf16", "e4m3"))} if form == "few" else {"z": rng.random() < 0.4})
    e = rng.choice((4, 8, 16, 48, 64, 160))
    k = rng.randint(1, min(8, e))
    if op == "tokens":
        form = rng.choice(("dispatch", "combine", "combine_grad"))
        t = _log(rng, 1, 65536 // k if form == "dispatch" else 8192)
        c = {"op": op, "form": form, "t": t, "d": 32 * _log(rng, 1, max(1, min(128, (1 << 22) // (t * k + 31 * e)))), "e": e,
             "k": k}
        if form == "dispatch":
            return c | {"align": rng.choice((1, 32)), "codes": rng.random() < 0.5}
        c |= {"align": rng.choice((1, 32)), "z": rng.choice(("bf16", "fp32"))}
        return c | ({"residual": rng.random() < 0.5} if form == "combine" else {"dy": rng.choice(("bf16", "fp32"))})
    form = rng.choice(("rows", "wgrad", "few"))
    c = {"op": op, "form": form, "t": _log(rng, 1, max(1, 256 // k) if form == "few" else 65536 // k),
         "n": 32 * _log(rng, 1, 64), "d": 32 * _log(rng, 1, 64), "e": min(e, 64), "k": k}
    if form == "few":
        return c | {"x": rng.choice(("bf16", "e4m3")), "gate": rng.random() < 0.5}
    return c | ({"out": rng.choice(("bf16", "fp32"))} if form == "rows" else {})


# ------------------------------------------------------------------ inputs


def capacity(slots, e, align):
    """Rows of the sorted buffers: every slot and the padding of every expert that can have one."""
    if align == 1:
        return slots
    return -(-(slots + min(e, slots) * (align - 1)) // 256) * 256


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


def _mxfp4(y):
    """(codes, scales) of fp32 rows: E2M1 values, two a byte, in blocks of 32 under upward E8M0 scales."""
    b = y.unflatten(-1, (-1, 32))
    e = _upward(b.abs().amax(-1), 6.0)
    v = (b * _pow2(-e)[..., None]).flatten(-2)
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda")
    code = torch.bucketize(v.abs(), mids, out_int32=True).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8)


def _weights(g, *shape):
    """N(0, 0.02) MXFP4 weights along the last axis, one expert at a time."""
    if len(shape) == 2:
        return _mxfp4(0.02 * torch.randn(shape, device="cuda", generator=g))
    parts = [_mxfp4(0.02 * torch.randn(shape[1:], device="cuda", generator=g)) for _ in range(shape[0])]
    return torch.stack([c for c, _ in parts]), torch.stack([s for _, s in parts])


def _routed(g, case):
    """(ids, weights) of a router: k experts a token, some experts liked better, the last 64th of a batch unrouted."""
    t, e, k = case["t"], case["e"], case["k"]
    score = torch.randn((t, e), device="cuda", generator=g) + 0.5 * torch.randn(e, device="cuda", generator=g)
    top, ids = score.topk(k, -1)
    ids = ids.int()
    if case["form"] != "few":
        ids[t - t // 64:] = -1
    w = torch.exp(top - top.amax(-1, keepdim=True))
    return ids, w / w.sum(-1, keepdim=True)


def _sorted(ids, e, align):
    """(offsets, slots, rows) of the sorted tokens, by counting the earlier slots of the same expert."""
    flat = ids.flatten()
    n, cap = flat.numel(), capacity(flat.numel(), e, align)
    hit = flat == torch.arange(e, device="cuda")[:, None]
    seen = hit.int().cumsum(-1)
    size = (seen[:, -1] + (align - 1)) // align * align
    offsets = torch.cat((size.new_zeros(1), size.cumsum(0)))
    routed = hit.any(0)
    at = flat.clamp(0, e - 1).long()
    row = offsets[at] + seen.gather(0, at[None])[0] - 1
    # unrouted slots write one place behind the end, which is cut off: nothing depends on the data's count
    slots = torch.full((cap + 1,), -1, dtype=torch.int32, device="cuda")
    slots[torch.where(routed, row, cap)] = torch.arange(n, dtype=torch.int32, device="cuda")
    return offsets.int(), slots[:cap].clone(), torch.where(routed, row, -1).int().reshape(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 29)
    op, form, s = case["op"], case["form"], {"case": case}
    kind = lambda x, name: x if name == "fp32" else x.bfloat16()  # noqa: E731
    if op == "act":
        m, n = case["m"], case["n"]
        if form == "grad":
            s["dy"] = kind(1e-3 * torch.randn((m, n), device="cuda", generator=g), case["dy"])
            s["z"] = (1.3 * torch.randn((m, n), device="cuda", generator=g)).bfloat16()
            return s
        x = _activations(g, m, case["d"])
        if form == "gemm":
            s["x"], s["x_scales"] = _mxfp4(x.bfloat16().float())
        elif case["x"] == "e4m3":
            s["x"], s["x_scales"] = (v.view(torch.uint8) for v in _e4m3(x))
        else:
            s["x"], s["x_scales"] = x.bfloat16(), None
        s["w"] = _weights(g, n, case["d"])
        s["bias"] = (0.1 * torch.randn(n, device="cuda", generator=g)).bfloat16() if case["bias"] else None
        s["residual"] = _activations(g, m, n).bfloat16() if case["residual"] else None
        return s
    ids, s["weights"] = _routed(g, case)
    t, d, e = case["t"], case["d"], case["e"]
    if op == "tokens":
        if form == "dispatch":
            return s | {"ids": ids, "x": _activations(g, t, d).bfloat16()}
        s["offsets"], s["slots"], s["rows"] = _sorted(ids, e, case["align"])
        z = torch.randn((s["slots"].numel(), d), device="cuda", generator=g) * (s["slots"] >= 0)[:, None]
        s["z"] = kind(z, case["z"])
        if form == "combine":
            s["residual"] = _activations(g, t, d).bfloat16() if case["residual"] else None
        else:
            s["dy"] = kind(1e-3 * torch.randn((t, d), device="cuda", generator=g), case["dy"])
        return s
    s["offsets"], s["slots"], rows = _sorted(ids, e, 1 if form == "few" else 32)
    s["segments"] = s["offsets"].tolist()  # of the plain forms, which walk the experts on the host
    token = s["slots"].clamp(min=0).long() // case["k"]
    stands = (s["slots"] >= 0)[:, None]
    x = (_activations(g, t, d)[token] * stands).bfloat16().float()
    if form == "wgrad":
        dy = (1e-3 * torch.randn((t, case["n"]), device="cuda", generator=g))[token] * stands
        s["a"], s["a_scales"] = _mxfp4(dy.bfloat16().float().t().contiguous())
        s["x"], s["x_scales"] = _mxfp4(x.t().contiguous())
        return s
    if form == "rows":
        s["x"], s["x_scales"] = _mxfp4(x)
    elif case["x"] == "e4m3":
        s["x"], s["x_scales"] = (v.view(torch.uint8) for v in _e4m3(x))
    else:
        s["x"], s["x_scales"] = x.bfloat16(), None
    s["w"] = _weights(g, e, case["n"] * (2 if case.get("gate") else 1), d)
    return s


def work(case):
    op, form, size = case["op"], case["form"], {"bf16": 2, "fp32": 4, "e4m3": 1 + 1 / 32}
    if op == "act":
        m, n = case["m"], case["n"]
        if form == "grad":
            return {"bytes": m * n * (size[case["dy"]] + 2 + 2) + 4 * n, "flops": 12 * m * n}
        d = case["d"]
        x = m * d * (size[case["x"]] if form == "few" else 17 / 32)
        y = m * n * (size[case["out"]] + 2 * case["residual"] + 2 * case.get("z", False)) + 2 * n * case["bias"]
        return {"bytes": x + n * d * 17 / 32 + y, "flops": 2 * m * n * d}
    t, d, e, slots = case["t"], case["d"], case["e"], case["t"] * case["k"]
    if op == "tokens":
        cap = capacity(slots, e, case["align"])
        index = 4 * (2 * slots + cap + e + 1)
        if form == "dispatch":
            return {"bytes": index + 2 * t * d + cap * d * (2 + (1 + 1 / 32) * case["codes"]), "flops": 2 * cap * d}
        if form == "combine":
            return {"bytes": 8 * slots + slots * d * size[case["z"]] + t * d * (2 + 2 * case["residual"]), "flops": 2 * slots * d}
        return {"bytes": 12 * slots + slots * d * size[case["z"]] + t * d * size[case["dy"]] + 2 * cap * d, "flops": 3 * slots * d}
    n = case["n"] * (2 if case.get("gate") else 1)
    hit = e * (1 - (1 - case["k"] / e) ** t)  # experts that a batch reaches, on average
    if form == "wgrad":
        return {"bytes": slots * (n + d) * 17 / 32 + 4 * e * n * d, "flops": 2 * slots * n * d}
    x = slots * d * (17 / 32 if form == "rows" else size[case["x"]])
    y = slots * case["n"] * (4 if form == "few" and not case["gate"] else size.get(case.get("out"), 2))
    return {"bytes": x + hit * n * d * 17 / 32 + y, "flops": 2 * slots * n * d}


# ------------------------------------------------------------------ plain forms


def _decoded(codes, scales):
    """fp32 values of E2M1 codes under E8M0 scales."""
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda")
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * scales.view(torch.float8_e8m0fnu).float()[..., None]).flatten(-2)


def _rows_of(st):
    """fp32 values of a few-row product's activations."""
    if st["x_scales"] is None:
        return st["x"].float()
    scale = st["x_scales"].view(torch.float8_e8m0fnu).float()
    return (st["x"].view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        sig = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return sig + z * sig * (1 - sig) * (c * (1 + 3 * 0.044715 * z * z))
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return torch.ones_like(z)


def _plain(st):
    case = st["case"]
    op, form = case["op"], case["form"]
    if op == "act":
        if form == "grad":
            dz = st["dy"].float() * _act_grad(st["z"].float(), case["act"])
            return {"dz": dz.bfloat16(), "dbias": dz.sum(0)}
        z = (_decoded(st["x"], st["x_scales"]) if form == "gemm" else _rows_of(st)) @ _decoded(*st["w"]).t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        y = y if case["out"] == "fp32" else y.bfloat16()
        return {"y": y, "z": z.bfloat16()} if case.get("z") else {"y": y}
    if op == "tokens":
        k = case["k"]
        if form == "dispatch":
            offsets, slots, rows = _sorted(st["ids"], case["e"], case["align"])
            xs = torch.where((slots >= 0)[:, None], st["x"][slots.clamp(min=0).long() // k], 0.0)
            out = {"offsets": offsets, "slots": slots, "rows": rows, "x": xs}
            return out | (dict(zip(("codes", "scales"), _e4m3(xs.float()))) if case["codes"] else {})
        routed, at = st["rows"] >= 0, st["rows"].clamp(min=0).long()
        if form == "combine":
            y = torch.zeros((case["t"], case["d"]), device="cuda")
            for j in range(k):
                y += torch.where(routed[:, j:j + 1], st["weights"][:, j:j + 1] * st["z"][at[:, j]].float(), 0.0)
            return (y if st["residual"] is None else y + st["residual"].float()).bfloat16()
        dy, slot = st["dy"].float(), st["slots"].clamp(min=0).long()
        dz = torch.where((st["slots"] >= 0)[:, None], st["weights"].flatten()[slot][:, None] * dy[slot // k], 0.0)
        dw = torch.stack([(dy * st["z"][at[:, j]].float()).sum(-1) for j in range(k)], -1)
        return {"dz": dz.bfloat16(), "dw": torch.where(routed, dw, 0.0)}
    seg, e, n = st["segments"], case["e"], case["n"]
    if form == "wgrad":
        a, b = _decoded(st["a"], st["a_scales"]), _decoded(st["x"], st["x_scales"])
        return torch.stack([a[:, seg[i]:seg[i + 1]] @ b[:, seg[i]:seg[i + 1]].t() for i in range(e)])
    x = _decoded(st["x"], st["x_scales"]) if form == "rows" else _rows_of(st)
    y = torch.zeros((x.shape[0], n * (2 if case.get("gate") else 1)), device="cuda")
    for i in range(e):
        if seg[i + 1] > seg[i]:
            y[seg[i]:seg[i + 1]] = x[seg[i]:seg[i + 1]] @ _decoded(st["w"][0][i], st["w"][1][i]).t()
    if not case.get("gate"):
        return y if case.get("out", "fp32") == "fp32" else y.bfloat16()
    a, b = y.bfloat16().float().chunk(2, -1)
    return (a / (1 + torch.exp(-a)) * b).bfloat16()


# ------------------------------------------------------------------ the package's calls


_package = None


def _own(st):
    global _package
    if _package is None:
        import precision_mxfp4_producers_amd
        _package = precision_mxfp4_producers_amd
    mx, case = _package, st["case"]
    op, form = case["op"], case["form"]
    if op == "act":
        act = ACTS.index(case["act"])
        if form == "grad":
            dz, dbias = mx.fp4_act_backward(st["dy"], st["z"], act)
            return {"dz": dz, "dbias": dbias}
        dtype = torch.float32 if case["out"] == "fp32" else torch.bfloat16
        if form == "few":
            return {"y": mx.fp4_matvec_act(st["x"], *st["w"], act, x_scales=st["x_scales"], bias=st["bias"],
                                           residual=st["residual"], dtype=dtype)}
        y, z = mx.fp4_gemm_act(st["x"], st["x_scales"], *st["w"], act, bias=st["bias"], residual=st["residual"], dtype=dtype,
                               emit_z=case["z"])
        return {"y": y, "z": z} if case["z"] else {"y": y}
    if op == "tokens":
        if form == "dispatch":
            offsets, slots, rows = mx.fp4_expert_sort(st["ids"], case["e"], case["align"])
            xs, codes, scales = mx.fp4_expert_gather(st["x"], slots, case["k"], fmt=mx.FP4_E4M3, emit_codes=case["codes"])
            out = {"offsets": offsets, "slots": slots, "rows": rows, "x": xs}
            return out | ({"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
                          if case["codes"] else {})
        if form == "combine":
            return mx.fp4_expert_combine(st["z"], st["rows"], st["weights"], residual=st["residual"])
        dz, dw = mx.fp4_expert_combine_backward(st["dy"], st["z"], st["slots"], st["rows"], st["weights"])
        return {"dz": dz, "dw": dw}
    if form == "wgrad":
        return mx.fp4_gemm_experts_wgrad(st["offsets"], st["a"], st["a_scales"], st["x"], st["x_scales"])
    if form == "rows":
        return mx.fp4_gemm_experts(st["offsets"], st["x"], st["x_scales"], *st["w"],
                                   dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    if case["gate"]:
        return mx.fp4_swiglu_matvec_experts(st["offsets"], st["x"], *st["w"], x_scales=st["x_scales"])
    return mx.fp4_matvec_experts(st["offsets"], st["x"], *st["w"], x_scales=st["x_scales"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64-bit values


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


def _values(codes, scales):
    w = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = _fp4_value(codes & 15), _fp4_value(codes >> 4)
    return w.mul_(_unit(scales.long() - 127).repeat_interleave(32, -1))


def _few_values(st):
    if st["x_scales"] is None:
        return st["x"].double()
    return _e4m3_value(st["x"]) * _unit(st["x_scales"].long() - 127).repeat_interleave(32, -1)


def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _tanh_arg(z):
    return math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3))


def exact(case, seed):
    st = prepare(case, seed)
    op, form = case["op"], case["form"]
    if op == "act":
        act = case["act"]
        if form == "grad":
            z = st["z"].double()
            if act == "none":
                s = torch.ones_like(z)
            elif act == "relu":
                s = (z > 0).double()
            elif act == "gelu":
                s = _phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
            elif act == "gelu_tanh":
                u = torch.tanh(_tanh_arg(z))
                s = 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
            else:
                s = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
            dz = s.mul_(st["dy"].double())
            return {"dz": dz, "dbias": dz.sum(0)}
        x = _values(st["x"], st["x_scales"]) if form == "gemm" else _few_values(st)
        z = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for at in range(0, case["n"], 4096):  # weights in parts: their 64-bit values take sixteen times the codes' room
            z[:, at:at + 4096] = x @ _values(st["w"][0][at:at + 4096], st["w"][1][at:at + 4096]).t()
        if st["bias"] is not None:
            z += st["bias"].double()
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "gelu": lambda: z * _phi(z),
             "gelu_tanh": lambda: z * torch.sigmoid(2 * _tanh_arg(z)), "silu": lambda: z * torch.sigmoid(z)}[act]()
        if st["residual"] is not None:
            y = y + st["residual"].double()
        return {"y": y, "z": z} if case.get("z") else {"y": y}
    e, k = case["e"], case["k"]
    if op == "tokens":
        if form == "dispatch":
            align, flat = case["align"], st["ids"].flatten().cpu()
            cap = capacity(flat.numel(), e, align)
            offsets, slots, rows = [0], torch.full((cap,), -1, dtype=torch.int32), torch.full_like(flat, -1)
            for i in range(e):
                mine = (flat == i).nonzero()[:, 0]
                at = offsets[-1]
                slots[at:at + len(mine)] = mine.int()
                rows[mine] = torch.arange(at, at + len(mine), dtype=torch.int32)
                offsets.append(at + -(-len(mine) // align) * align)
            slots = slots.cuda()
            xs = torch.zeros((cap, case["d"]), dtype=torch.float64, device="cuda")
            xs[slots >= 0] = st["x"].double()[slots[slots >= 0].long() // k]
            out = {"offsets": torch.tensor(offsets, dtype=torch.int32).cuda(), "slots": slots,
                   "rows": rows.reshape(st["ids"].shape).cuda(), "x": xs}
            if not case["codes"]:
                return out
            b = xs.reshape(cap, -1, 32)
            top = b.abs().max(-1).values
            # the smallest e with 448 2^e >= top: the exponent of top / 448, or one below where that is a power of two
            ex = torch.frexp(top / 448).exponent
            ex = torch.where(448 * _unit(ex - 1) >= top, ex - 1, ex)
            ex = torch.where(top > 0, ex, -127)
            q = b / _unit(ex).unsqueeze(-1)
            step = _unit(torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent - 4)
            return out | {"codes": (torch.round(q / step) * step).reshape(cap, case["d"]), "scales": _unit(ex)}
        rows, w = st["rows"].long(), st["weights"].double()
        hit = (rows >= 0).double()
        if form == "combine":
            y = torch.zeros((case["t"], case["d"]), dtype=torch.float64, device="cuda")
            for j in range(k):
                y += (w[:, j] * hit[:, j])[:, None] * st["z"][rows[:, j]].double()
            return y if st["residual"] is None else y + st["residual"].double()
        dy = st["dy"].double()
        dz = torch.zeros((st["slots"].numel(), case["d"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for j in range(k):
            own_rows = rows[:, j][rows[:, j] >= 0]
            dz[own_rows] = (w[:, j, None] * dy)[rows[:, j] >= 0]
            dw[:, j] = (dy * st["z"][rows[:, j]].double()).sum(-1) * hit[:, j]
        return {"dz": dz, "dw": dw}
    seg, n = st["segments"], case["n"]
    if form == "wgrad":
        out = torch.zeros((e, n, case["d"]), dtype=torch.float64, device="cuda")
        a, b = _values(st["a"], st["a_scales"]), _values(st["x"], st["x_scales"])
        for i in range(e):
            out[i] = torch.mm(a[:, seg[i]:seg[i + 1]], b[:, seg[i]:seg[i + 1]].t())
        return out
    x = _values(st["x"], st["x_scales"]) if form == "rows" else _few_values(st)
    y = torch.zeros((x.shape[0], st["w"][0].shape[1]), dtype=torch.float64, device="cuda")
    for i in range(e):
        y[seg[i]:seg[i + 1]] = torch.mm(x[seg[i]:seg[i + 1]], _values(st["w"][0][i], st["w"][1][i]).t())
    if not case.get("gate"):
        return y
    a, b = _rounded(y[:, :n]), _rounded(y[:, n:])
    return a * torch.sigmoid(a) * b
