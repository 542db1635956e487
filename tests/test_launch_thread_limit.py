"""Sizes whose launch would have 2^32 threads or more in one dimension are refused by
the calls that launch one: such a launch wraps, with no error.  No GPU needed: the
refusal comes before anything is enqueued, and the pointers are never read."""

import ctypes

import pytest

import precision_mxfp4_producers_amd as mx

V, I = ctypes.c_void_p, ctypes.c_int64
ESHAPE = 2


@pytest.fixture(scope="module")
def lib():
    return mx.load()


def test_quantizers(lib):
    p = V(4096)
    n = 1 << 35                                            # one row: 2^24 workgroups of 256 threads, eight values each
    assert lib.fp4_quantize_rows(p, 1, n, n, p, p, 0, 0, 0, None) == ESHAPE
    assert lib.fp4_quantize_rows(p, 1, n - 2016, n, p, p, 1, 0, 0, None) == ESHAPE
    assert lib.fp4_nv_quantize_rows(p, 1, n, n, p, p, p, p, 0, 0, 0, None) == ESHAPE
    assert lib.fp4_swiglu_backward(32, n, p, n, p, p, p, p, None) == ESHAPE
    n = 1 << 31                                            # 2^24 strips of 128 columns
    assert lib.fp4_quantize_cols(p, 32, n, n, p, p, 32, 0, None) == ESHAPE
    assert lib.fp4_quantize_dual(p, 32, n, n, p, p, 0, 0, 0, p, p, 32, 0, None) == ESHAPE
    assert lib.fp4_quantize_dual(p, 32, n - 224, n, p, p, 0, 0, 0, p, p, 32, 0, None) == ESHAPE


@pytest.mark.parametrize("m,n,k", [(32, 1 << 31, 256), (1 << 31, 32, 512), (1 << 19, 1 << 20, 256), (32, 1 << 32, 32), (1 << 20, 1 << 20, 288)])
def test_products(lib, m, n, k):
    p = V(4096)
    assert lib.fp4_gemm(m, n, k, p, p, p, p, p, n, 0, None) == ESHAPE
    assert lib.fp4_gemm_pair(m, n, k, *[p] * 9, n, 0, None) == ESHAPE
    if k % 64 == 0 and k == 256:
        assert lib.fp4_nv_gemm(m, n, k, p, p, p, 1, p, p, p, 1, p, n, 0, None) == ESHAPE


def test_fill_of_an_empty_reduction(lib):
    n = 1 << 32
    assert lib.fp4_gemm(32, n, 0, None, None, None, None, V(4096), n, 0, None) == ESHAPE


def test_products_together(lib):
    p = 4096
    P = mx._GemmProblem
    n = 1 << 30                                            # 2^22 tiles each, 2^23 together
    arr = (P * 2)(*[P(32, n, 256, p, p, p, p, None, None, None, None, p, n, 0)] * 2)
    assert lib.fp4_gemm_grouped(ctypes.cast(arr, V), 2, None) == ESHAPE


def test_gated(lib):
    p = V(4096)
    for t, f, d in ((1 << 31, 32, 256), (32, 1 << 30, 0), (32, 1 << 31, 32), (1 << 20, 1 << 19, 512)):
        assert lib.fp4_swiglu_producer(t, f, d, *[p] * 10, 0, None) == ESHAPE
    assert lib.fp4_gemm_swiglu_backward_producer(1 << 31, 32, 256, *[p] * 6, 0, 0, 0, 0, *[p] * 8, None) == ESHAPE
