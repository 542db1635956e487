"""The README's two sequences of the expert and epilogue calls: each result the
right product of its bf16 inputs (relative L2 error of MXFP4 size, where a
transposed or mismatched operand gives an error near 1.4)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def near(got, want, bound):
    assert got.shape == want.shape
    rel = float((got.double() - want).norm() / want.norm())
    assert rel < bound, f"relative L2 error {rel:.3f}"


def silu(a):
    return a * torch.sigmoid(a)


def test_epilogue_usage(gpu_lib):
    mx = gpu_lib
    T, D, N = 512, 256, 384
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, D, device="cuda", generator=g).bfloat16()
    w = (0.1 * torch.randn(N, D, device="cuda", generator=g)).bfloat16()
    dy = torch.randn(T, N, device="cuda", generator=g).bfloat16()
    bias = torch.randn(N, device="cuda", generator=g)
    xr, xrs = mx.fp4_quantize_rows(x)
    wr, wrs = mx.fp4_quantize_w2d32(w)[:2]
    h, z = mx.fp4_gemm_act(xr, xrs, wr, wrs, mx.FP4_ACT_GELU, bias=bias, emit_z=True)
    dz, dbias = mx.fp4_act_backward(dy, z, mx.FP4_ACT_GELU)
    h1 = mx.fp4_matvec_act(x[:1], wr, wrs, mx.FP4_ACT_GELU, bias=bias)
    z64 = (x.double() @ w.double().T + bias.double()).requires_grad_()
    h64 = torch.nn.functional.gelu(z64)
    dz64, = torch.autograd.grad(h64, z64, dy.double())
    near(z, z64.detach(), 0.3)
    near(h, h64.detach(), 0.3)
    near(h1, h64[:1].detach(), 0.3)
    near(dz, dz64, 0.3)
    near(dbias, dz64.sum(0), 0.3)


def test_layer_of_experts_usage(gpu_lib):
    mx = gpu_lib
    T, D, E, k, F = 512, 256, 8, 2, 320
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s, std=1.0: (std * torch.randn(*s, device="cuda", generator=g)).bfloat16()  # noqa: E731
    x, dy = rand(T, D), rand(T, D, std=1e-3)
    w1f, w3f, w2f = rand(E, F, D, std=0.1), rand(E, F, D, std=0.1), rand(E, D, F, std=0.1)
    mask = mx.fp4_sign_mask_from_seed(0)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k).indices
    weights = torch.rand(T, k, device="cuda", generator=g)
    w1, w3, w2 = ([torch.stack(v) for v in zip(*(mx.fp4_quantize_w2d32(w) for w in ws))] for ws in (w1f, w3f, w2f))
    w13 = [torch.cat((w1[i], w3[i]), 1) for i in range(2)]

    off, slots, rows = mx.fp4_expert_sort(ids, E)
    xs, xsc, xss = mx.fp4_expert_gather(x, slots, k)
    xst, xsts = mx.fp4_quantize_cols(xs, 32, mask)
    a, b, hc, hs, htc, hts = mx.fp4_swiglu_producer_experts(off, xsc, xss, *w13, mask)
    zs = mx.fp4_gemm_experts(off, hc, hs, *w2[:2], dtype=torch.bfloat16)
    out = mx.fp4_expert_combine(zs, rows, weights, residual=x)

    dzs, dweights = mx.fp4_expert_combine_backward(dy, zs, slots, rows, weights)
    dr, drs, dc, dcs = mx.fp4_quantize_dual(dzs, mx.FP4_SR, 1234, 1, 32, mask)
    dw2 = mx.fp4_gemm_experts_wgrad(off, dc, dcs, htc, hts)
    dh = mx.fp4_gemm_experts(off, dr, drs, *w2[2:])
    (ar, ars), (br, brs), (ac, acs), (bc, bcs) = mx.fp4_swiglu_backward_producer(dh, a, b, 1234, 2, 3, mask)
    dw1 = mx.fp4_gemm_experts_wgrad(off, ac, acs, xst, xsts)
    dw3 = mx.fp4_gemm_experts_wgrad(off, bc, bcs, xst, xsts)
    dxs = mx.fp4_gemm_experts(off, ar, ars, *w1[2:], dtype=torch.bfloat16, pair=(br, brs, *w3[2:]))
    dx = mx.fp4_expert_combine(dxs, rows)

    off, slots, rows = mx.fp4_expert_sort(ids[:1], E, align=1)
    x1, _, _ = mx.fp4_expert_gather(x[:1], slots, k, emit_codes=False)
    h1 = mx.fp4_swiglu_matvec_experts(off, x1, *w13)
    out1 = mx.fp4_expert_combine(mx.fp4_matvec_experts(off, h1, *w2[:2]), rows, weights[:1], residual=x[:1])

    # the dense form on the CPU in 64 bits: every expert on every token, weighted
    xd, p1, p3, p2, wd = (v.double().cpu().requires_grad_() for v in (x, w1f, w3f, w2f, weights))
    gate = torch.zeros(T, E, dtype=torch.float64).scatter_add(1, ids.cpu(), wd)
    branch = sum(gate[:, e:e + 1] * ((silu(xd @ p1[e].T) * (xd @ p3[e].T)) @ p2[e].T) for e in range(E))
    grads = torch.autograd.grad(branch, (xd, p1, p3, p2, wd), dy.double().cpu())
    want = (branch + xd).detach()
    near(out.cpu(), want, 0.5)
    near(out1.cpu(), want[:1], 0.5)
    for got, ref in zip((dx, dw1, dw3, dw2, dweights), grads):
        near(got.cpu(), ref, 0.6)
