"""Codes that the sorted rows' producers leave: the gated producer's against its own a
and b byte for byte for every row length, the gather's of rows that hold infinities and
NaN, and few-row products where a router sends nearly all rows to one expert."""

import numpy as np
import pytest
import torch

import synthetic
from oracle import experts as X
from oracle import formats as F
from oracle import gemm as G
from oracle import norm as N
from oracle import quant as Q
from oracle import swiglu as S
from test_gpu_experts import MANY_ROWS, bf16, choices
from test_gpu_gemm_experts import SWIGLU, check, check_gate, codes, dev, host, segments

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra", [0, 32, 320])
@pytest.mark.parametrize("sizes,f,d", SWIGLU + [((1, 700, 33), 416, 1056), ((40, 3), 128, 4096 + 32)])
def test_gated_producer(gpu_lib, sizes, f, d, extra):
    """a and b against float64; h, quantized both ways, from those a and b."""
    offsets, rows = segments(sizes, 32)
    rows += extra
    if rows == 0:
        return
    x, mask = codes((rows, d), 1), gpu_lib.fp4_sign_mask_from_seed(3)
    w = [Q.quantize_w2d32(synthetic.tensor((2 * f, d), std=0.05, seed=10 + i), 0.87)[:2] for i in range(len(sizes))]
    wc, ws = np.stack([c for c, _ in w]), np.stack([s for _, s in w])
    a, b, hc, hs, htc, hts = gpu_lib.fp4_swiglu_producer_experts(dev(offsets), *map(dev, x), dev(wc), dev(ws), mask)
    ref, e = np.zeros((2, rows, 2 * f))
    for i in range(len(sizes)):
        at = slice(offsets[i], offsets[i + 1])
        ref[at], e[at] = G.gemm_ref(x[0][at], x[1][at], wc[i], ws[i])
    check(a.view(torch.bfloat16), ref[:, :f], e[:, :f], d, f32=False)
    check(b.view(torch.bfloat16), ref[:, f:], e[:, f:], d, f32=False)
    h = S.swiglu_h(host(a.view(torch.int16)).view(np.uint16), host(b.view(torch.int16)).view(np.uint16))
    want = (*Q.quantize_rows(h), *Q.quantize_cols(h, 32, mask))
    for got, v, name in zip((hc, hs, htc, hts), want, ("row codes", "row scales", "column codes", "column scales")):
        assert np.array_equal(host(got), v), name


@pytest.mark.parametrize("t,k,e,d,align", [(130, 3, 7, 1056, 32), (65, 2, 4, 96, 1), MANY_ROWS[0]])
def test_gather_of_rows_without_numbers(gpu_lib, t, k, e, d, align):
    """Infinities and NaN go out bit for bit; the E2M1 codes are those of the row
    quantizer, and of the other rows those of the same tensor without them."""
    x = synthetic.tensor((t, d), seed=d)
    _, slots, _ = X.sort(choices(t, k, e, d, "holes"), e, align)
    plain = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), k)
    plain8 = gpu_lib.fp4_expert_gather(bf16(x), dev(slots), k, fmt=gpu_lib.FP4_E4M3)
    odd = np.arange(0, t, 5)
    y = x.copy()
    for i, r in enumerate(odd):
        y[r, (37 * i) % d] = (0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x7F81)[i % 5]
    y[odd[0]] = 0x7FFF
    xs, qc, qs = gpu_lib.fp4_expert_gather(bf16(y), dev(slots), k)
    want = X.gather(y, slots, k)
    assert np.array_equal(host(xs.view(torch.int16)).view(np.uint16), want)
    wc, ws = gpu_lib.fp4_quantize_rows(xs)
    assert torch.equal(qc, wc) and torch.equal(qs, ws)
    xs8, qc8, qs8 = gpu_lib.fp4_expert_gather(bf16(y), dev(slots), k, fmt=gpu_lib.FP4_E4M3)
    assert torch.equal(xs8.view(torch.int16), xs.view(torch.int16))
    rest = dev(np.nonzero(~((slots >= 0) & np.isin(slots // k, odd)))[0])
    for got, was in ((qc, plain[1]), (qs, plain[2]), (qc8, plain8[1]), (qs8, plain8[2])):
        assert torch.equal(got[rest], was[rest])


CROWDED = [((170,) + (0, 1) * 31 + (2,), 96, 512), ((0, 0, 190, 1, 0, 1), 300, 1056), ((1, 400), 33, 8192), ((64,) * 2 + (0,) * 1000 + (1, 1), 16, 128)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("sizes,n,k", CROWDED)
def test_few_row_products_of_a_crowded_expert(gpu_lib, sizes, n, k, kind):
    offsets, rows = segments(sizes, 1)
    bits = synthetic.tensor((rows, k), seed=k)
    x64, x, scales = F.bf16_bits_to_f64(bits), bf16(bits), None
    if kind == "e4m3":
        c, s = N.encode_e4m3(bits)
        x64, x, scales = N.decode_e4m3(c, s), dev(c), dev(s)
    w = codes((len(sizes), 2 * n, k), 2)
    got = gpu_lib.fp4_matvec_experts(dev(offsets), x, *map(dev, w), x_scales=scales)
    h = gpu_lib.fp4_swiglu_matvec_experts(dev(offsets), x, *map(dev, w), x_scales=scales)
    ref, e = np.zeros((2, rows, 2 * n))
    for i in np.nonzero(sizes)[0]:
        at, wi = slice(offsets[i], offsets[i + 1]), F.decode(w[0][i], w[1][i])
        ref[at], e[at] = x64[at] @ wi.T, abs(x64[at]) @ abs(wi).T
        for lo in range(offsets[i], offsets[i + 1], 64):
            part = slice(lo, min(lo + 64, offsets[i + 1]))
            want = gpu_lib.fp4_swiglu_matvec(x[part], dev(w[0][i]), dev(w[1][i]), x_scales=None if scales is None else scales[part])
            check_gate(h[part], want, x64[part], wi)
    check(got, ref, e, k)
