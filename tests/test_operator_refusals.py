"""The norm, dropout and few-row product calls answer invalid arguments, empty
shapes and sizes beyond their limits from the host checks (no GPU)."""

import ctypes

import pytest

OK, EINVAL, ESHAPE, EALIGN = 0, 1, 2, 3
P, ODD = 4096, 4097                                        # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import precision_mxfp4_producers_amd as mx
    return mx.load()


def call(fn, defaults, **changes):
    assert not set(changes) - set(defaults), changes
    return fn(*(defaults | changes).values())


DROPOUT = dict(rows=4, cols=40, x=P, xt=0, ldx=40, res=P, ldr=40, p=0.1, seed=0, offset=0, out=P, ldo=40, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(xt=2), EINVAL), (dict(p=-0.1), EINVAL), (dict(p=1.5), EINVAL), (dict(p=float("nan")), EINVAL),
    (dict(x=None), EINVAL), (dict(out=None), EINVAL),
    (dict(rows=-1), ESHAPE), (dict(cols=-1), ESHAPE), (dict(ldx=39), ESHAPE), (dict(ldr=39), ESHAPE),
    (dict(ldo=39), ESHAPE), (dict(rows=1 << 62), ESHAPE),
    (dict(cols=1 << 40, ldx=1 << 40, ldr=1 << 40, ldo=1 << 40), ESHAPE),
    (dict(x=ODD), EALIGN), (dict(res=ODD), EALIGN), (dict(out=ODD), EALIGN), (dict(xt=1, x=P + 2), EALIGN),
    (dict(rows=0, x=None, out=None), OK), (dict(cols=0, x=None, out=None), OK),
])
def test_dropout(lib, changes, want):
    assert call(lib.fp4_dropout, DROPOUT, **changes) == want


NORM = dict(t=4, d=64, x=P, xt=0, ldx=64, res=P, ldr=64, gamma=P, eps=1e-5, p=0.1, seed=0, offset=0, sum=P, rstd=P, y=P,
            fmt=1, codes=P, scales=P, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(xt=-1), EINVAL), (dict(fmt=2), EINVAL), (dict(p=2.0), EINVAL), (dict(p=float("nan")), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(x=None), EINVAL), (dict(gamma=None), EINVAL),
    (dict(rstd=None), EINVAL),
    (dict(t=-1), ESHAPE), (dict(t=1 << 31), ESHAPE), (dict(d=48), ESHAPE), (dict(d=-32), ESHAPE), (dict(ldx=32), ESHAPE),
    (dict(ldr=32), ESHAPE), (dict(d=32800, ldx=32800, ldr=32800), ESHAPE),
    (dict(x=P + 8), EALIGN), (dict(res=P + 8), EALIGN), (dict(gamma=P + 8), EALIGN), (dict(sum=P + 8), EALIGN),
    (dict(y=P + 8), EALIGN), (dict(codes=P + 8), EALIGN), (dict(rstd=P + 2), EALIGN), (dict(ldx=68), EALIGN),
    (dict(ldr=68), EALIGN), (dict(xt=1, ldx=66), EALIGN),
    (dict(t=0, x=None, gamma=None, rstd=None), OK), (dict(d=0, x=None, gamma=None, rstd=None), OK),
])
def test_rmsnorm_producer(lib, changes, want):
    assert call(lib.fp4_rmsnorm_producer, NORM, **changes) == want


BWD = dict(t=4, d=64, dy=P, dyt=1, lddy=64, s=P, lds=64, rstd=P, gamma=P, ds=P, ldds=64, p=0.1, seed=0, offset=0, dsum=P,
           dx=P, dgamma=P, accumulate=0, ws=P, size=1 << 20, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(dyt=2), EINVAL), (dict(p=-1.0), EINVAL), (dict(accumulate=2), EINVAL),
    *((dict([(n, None)]), EINVAL) for n in ("dy", "s", "rstd", "gamma", "dsum", "dx", "dgamma", "ws")),
    (dict(t=-1), ESHAPE), (dict(d=40), ESHAPE), (dict(lddy=32), ESHAPE), (dict(lds=32), ESHAPE), (dict(ldds=32), ESHAPE),
    (dict(t=1 << 31), ESHAPE), (dict(size=64 * 4 - 1), ESHAPE), (dict(d=32800, lddy=32800, lds=32800, ldds=32800), ESHAPE),
    *((dict([(n, P + 8)]), EALIGN) for n in ("dy", "s", "gamma", "ds", "dsum", "dx", "ws")),
    (dict(rstd=P + 2), EALIGN), (dict(dgamma=P + 2), EALIGN), (dict(lds=68), EALIGN), (dict(ldds=68), EALIGN),
    (dict(lddy=66), EALIGN), (dict(dyt=0, lddy=68), EALIGN),
    (dict(d=0, dy=None, dgamma=None, ws=None), OK),
])
def test_rmsnorm_backward(lib, changes, want):
    assert call(lib.fp4_rmsnorm_backward, BWD, **changes) == want


def test_rmsnorm_backward_workspace(lib):
    size = lib.fp4_rmsnorm_backward_workspace
    assert size(0, 64) == 0 and size(3, 64) == 64 * 4 and size(10 ** 9, 32768) == 512 * 32768 * 4
    assert size(-1, 64) == size(1, 33) == size(1, 32800) == size(1, -32) == -1


MATVEC = dict(m=3, n=5, k=64, x=P, ldx=64, xs=None, codes=P, scales=P, c=P, ldc=5, accumulate=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(accumulate=2), EINVAL), (dict(x=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(c=None), EINVAL),
    (dict(m=-1), ESHAPE), (dict(m=65), ESHAPE), (dict(n=-1), ESHAPE), (dict(k=48), ESHAPE), (dict(k=-32), ESHAPE),
    (dict(k=1 << 24, ldx=1 << 24), ESHAPE), (dict(ldx=1 << 24), ESHAPE), (dict(ldx=56), ESHAPE), (dict(ldc=4), ESHAPE),
    (dict(xs=P, ldx=72), ESHAPE), (dict(n=1 << 40, ldc=1 << 40), ESHAPE),
    (dict(x=P + 8), EALIGN), (dict(codes=P + 8), EALIGN), (dict(ldx=68), EALIGN), (dict(c=P + 2), EALIGN),
    (dict(m=0, x=None, c=None), OK), (dict(n=0, x=None, codes=None, c=None), OK),
    (dict(k=0, ldx=0, x=None, codes=None, scales=None, accumulate=1), OK),
])
def test_matvec(lib, changes, want):
    assert call(lib.fp4_matvec, MATVEC, **changes) == want


NV = dict(m=3, n=5, k=64, x=P, ldx=64, codes=P, scales=P, factors=P, stride=0, c=P, ldc=5, accumulate=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(accumulate=-1), EINVAL), (dict(stride=-1), EINVAL), (dict(factors=None), EINVAL), (dict(x=None), EINVAL),
    (dict(m=65), ESHAPE), (dict(k=16), ESHAPE), (dict(ldc=4), ESHAPE),
    (dict(factors=P + 2), EALIGN), (dict(c=P + 1), EALIGN), (dict(m=0), OK),
])
def test_nv_matvec(lib, changes, want):
    assert call(lib.fp4_nv_matvec, NV, **changes) == want


SWIGLU = dict(m=3, f=5, d=64, x=P, ldx=64, xs=None, codes=P, scales=P, h=P, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(x=None), EINVAL), (dict(codes=None), EINVAL), (dict(h=None), EINVAL), (dict(m=65), ESHAPE), (dict(f=-1), ESHAPE),
    (dict(d=40), ESHAPE), (dict(xs=P, ldx=72), ESHAPE), (dict(x=P + 4), EALIGN), (dict(h=ODD), EALIGN),
    (dict(m=0), OK), (dict(f=0), OK),
])
def test_swiglu_matvec(lib, changes, want):
    assert call(lib.fp4_swiglu_matvec, SWIGLU, **changes) == want
