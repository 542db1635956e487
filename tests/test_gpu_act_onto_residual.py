"""Few-row products with an epilogue written over their residual, as the header allows:
every split of K, rows of x staged or not, rows of the residual at a pitch."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 33, 32), (1, 4096, 4096), (5, 300, 1056), (16, 130, 14336), (64, 515, 2048), (3, 40, 0)])
def test_onto_the_residual(gpu_lib, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((m, k), device="cuda", generator=g).bfloat16()
    w = [torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g),
         torch.randint(118, 124, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)]
    bias, buf = torch.randn(n, device="cuda", generator=g), torch.randn((m, n + 5), device="cuda", generator=g).bfloat16()
    res, beside = buf[:, :n], buf[:, n:].clone()
    want = gpu_lib.fp4_matvec_act(x, *w, gpu_lib.FP4_ACT_GELU, bias=bias, residual=res)
    assert gpu_lib.fp4_matvec_act(x, *w, gpu_lib.FP4_ACT_GELU, bias=bias, residual=res, y=res) is res
    assert torch.equal(res, want) and torch.equal(buf[:, n:], beside)
