"""GELU and its slope far out on the negative side, relative to their own size.

Bounds: the fit of the normal tail is within 8e-5 of it up to 8 and 3e-4 up to 13 for
fp32 results, so 2^-13 and 2^-11; within 1e-3 (2^-9.9) for those rounded to bf16, and
a rounding is 2^-8.  Results below 2^-126 may be off by 2^-134, half the smallest bf16,
by the fit, and by as much in their rounding."""

import numpy as np
import pytest
import torch

from oracle import act as A
from oracle import formats as F
from test_gpu_act import dev, host

pytestmark = pytest.mark.gpu
H = 2.0 ** -8


def gelu(lib, bias, m, n, dtype, few):
    """GELU of `bias` [n], put into z by the bias of an empty product."""
    if few:
        x, w = torch.zeros((m, 0), device="cuda").bfloat16(), [torch.zeros((n, 0), dtype=torch.uint8, device="cuda")] * 2
        return lib.fp4_matvec_act(x, *w, A.GELU, bias=bias, dtype=dtype)
    empty = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((m, 0), (m, 0), (n, 0), (n, 0))]
    return lib.fp4_gemm_act(*empty, A.GELU, bias=bias, dtype=dtype)[0]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", ["few", "small tiles", "large tiles"])
def test_gelu_over_every_bf16(gpu_lib, rows, f32):
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    z = F.bf16_bits_to_f64(bits)
    fine = np.isfinite(z) & (np.abs(z) < 1e3)
    m = {"few": 1, "small tiles": 1, "large tiles": 300}[rows]
    got = host(gelu(gpu_lib, dev(bits.view(np.int16)).view(torch.bfloat16), m, 65536, torch.float32 if f32 else torch.bfloat16,
                    rows == "few"))
    want = A.value(np.where(fine, z, 0), A.GELU)
    fit = np.where(z >= -8, 2.0 ** -13, 2.0 ** -11)
    if f32:
        tol = fit * np.abs(want) + 2.0 ** -134
    else:
        fit = fit if rows == "few" else 2.0 ** -9.9
        tol = (H + (1 + H) * fit) * np.abs(want) + 2.0 ** -133
    bad = (np.abs(got - want) > tol) & fine
    assert not bad.any(), [(z[i], got[0, i], want[i]) for i in np.nonzero(bad.any(0))[0][:3]]


def test_gelu_of_normal_values(gpu_lib):
    """The 2-norm of fp32 results: the fit's 5.2e-8 and the exponential's last bit, twice."""
    z = np.random.default_rng(0).normal(size=1 << 20).astype(np.float32)
    got = host(gelu(gpu_lib, dev(z), 1, z.size, torch.float32, False))[0]
    want = A.value(z, A.GELU)
    assert np.linalg.norm(got - want) <= 1.1e-7 * np.linalg.norm(want)


def test_slope_of_gelu_far_out(gpu_lib):
    """Below -3 the slope is z times the density and a tenth of it or less the tail:
    within 2^-12, and a rounding."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    zt = dev(bits.view(np.int16)).view(torch.bfloat16).reshape(2048, 32)
    got = host(gpu_lib.fp4_act_backward(torch.ones((2048, 32), device="cuda"), zt, A.GELU, emit_dbias=False)[0])
    z = host(zt).astype(np.float64)
    out = (z <= -3) & (z > -100)
    want = A.slope(np.where(out, z, 0), A.GELU)
    assert (np.abs(got - want) <= (H + 2.0 ** -12) * np.abs(want) + 2.0 ** -133)[out].all()
