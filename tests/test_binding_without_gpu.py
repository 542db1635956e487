"""The binding refuses host tensors by name, also where no GPU is visible."""

import pytest
import torch

import precision_mxfp4_producers_amd as mx

X, G, R = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16), torch.ones(4)
W, S, S4, F = (torch.zeros(6, n, dtype=torch.uint8) for n in (32, 2, 4, 1))

CALLS = [
    (lambda: mx.fp4_quantize_rows(X), "x"),
    (lambda: mx.fp4_dropout(X, 0.1), "x"),
    (lambda: mx.fp4_dropout([1.0], 0.1), "x"),
    (lambda: mx.fp4_rmsnorm_producer(X, G), "x"),
    (lambda: mx.fp4_rmsnorm_backward(X, X, R, G), "dy"),
    (lambda: mx.fp4_matvec(X, W, S), "x"),
    (lambda: mx.fp4_matvec(None, W, S), "x"),
    (lambda: mx.fp4_nv_matvec(X, W, S4, torch.ones(1)), "x"),
    (lambda: mx.fp4_swiglu_matvec(X, W, S), "x"),
]


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_host_tensors_are_refused_by_name(call):
    fn, name = CALLS[call]
    with pytest.raises(mx.Fp4Error, match=f"^{name} must be a CUDA"):
        fn()
