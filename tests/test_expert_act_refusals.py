"""The expert and epilogue calls answer invalid arguments, empty shapes and sizes
beyond their limits from the host checks (no GPU)."""

import pytest
import torch

OK, EINVAL, ESHAPE, EALIGN = 0, 1, 2, 3
P, ODD = 4096, 4097                                        # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import precision_mxfp4_producers_amd as mx
    return mx.load()


def call(fn, defaults, **changes):
    assert not set(changes) - set(defaults), changes
    return fn(*(defaults | changes).values())


def each(names, value, want):
    return [(dict([(n, value)]), want) for n in names]


GEMM = dict(m=5, n=64, k=96, ac=P, asc=P, bc=P, bsc=P, bias=P, bt=0, act=2, res=P, ldr=64, z=P, y=P, yt=0, ldy=64, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(bt=2), EINVAL), (dict(yt=-1), EINVAL), (dict(act=5), EINVAL), (dict(act=-1), EINVAL),
    *each(("ac", "asc", "bc", "bsc", "y"), None, EINVAL),
    (dict(m=-1), ESHAPE), (dict(n=48), ESHAPE), (dict(n=-32), ESHAPE), (dict(k=40), ESHAPE), (dict(k=-32), ESHAPE),
    (dict(k=1 << 24), ESHAPE), (dict(ldy=56), ESHAPE), (dict(ldr=56), ESHAPE), (dict(m=1 << 62), ESHAPE),
    (dict(n=1 << 50, ldy=1 << 50, ldr=1 << 50), ESHAPE),
    *each(("ac", "asc", "bc", "bsc", "res", "z", "y"), P + 8, EALIGN), (dict(bias=ODD), EALIGN), (dict(bt=1, bias=P + 2), EALIGN),
    (dict(ldr=68), EALIGN), (dict(ldy=68), EALIGN), (dict(yt=1, ldy=66), EALIGN),
    (dict(m=0, ac=None, y=None), OK), (dict(n=0, ldy=0, ldr=0, y=None), OK),
])
def test_gemm_act(lib, changes, want):
    assert call(lib.fp4_gemm_act, GEMM, **changes) == want


FEW = dict(m=3, n=5, k=64, x=P, ldx=64, xs=None, codes=P, scales=P, bias=P, bt=0, act=4, res=P, ldr=5, y=P, yt=0, ldy=5, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(bt=2), EINVAL), (dict(yt=2), EINVAL), (dict(act=5), EINVAL), *each(("x", "codes", "scales", "y"), None, EINVAL),
    (dict(m=-1), ESHAPE), (dict(m=65), ESHAPE), (dict(n=-1), ESHAPE), (dict(k=48), ESHAPE), (dict(k=1 << 24, ldx=1 << 24), ESHAPE),
    (dict(ldx=56), ESHAPE), (dict(ldy=4), ESHAPE), (dict(ldr=4), ESHAPE), (dict(xs=P, ldx=72), ESHAPE),
    (dict(x=P + 8), EALIGN), (dict(codes=P + 8), EALIGN), (dict(ldx=68), EALIGN), (dict(y=ODD), EALIGN), (dict(yt=1, y=P + 2), EALIGN),
    (dict(res=ODD), EALIGN), (dict(bias=ODD), EALIGN), (dict(bt=1, bias=P + 2), EALIGN),
    (dict(m=0, x=None, y=None), OK), (dict(n=0, codes=None, y=None), OK),
])
def test_matvec_act(lib, changes, want):
    assert call(lib.fp4_matvec_act, FEW, **changes) == want


BACK = dict(m=300, n=64, dy=P, dyt=1, lddy=64, z=P, ldz=64, act=2, dz=P, dbias=P, accumulate=0, ws=P, size=1 << 20, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(dyt=2), EINVAL), (dict(act=5), EINVAL), (dict(accumulate=2), EINVAL), *each(("dy", "z", "dz", "ws"), None, EINVAL),
    (dict(m=-1), ESHAPE), (dict(m=(1 << 40) + 1), ESHAPE), (dict(n=48), ESHAPE), (dict(n=(1 << 28) + 32, lddy=1 << 30, ldz=1 << 30), ESHAPE),
    (dict(lddy=56), ESHAPE), (dict(ldz=56), ESHAPE), (dict(size=0), ESHAPE),
    *each(("dy", "z", "dz", "ws"), P + 8, EALIGN), (dict(dbias=P + 2), EALIGN), (dict(ldz=68), EALIGN), (dict(lddy=66), EALIGN),
    (dict(dyt=0, lddy=68), EALIGN),
    (dict(n=0, dy=None, dbias=None), OK), (dict(m=0, dbias=None, dy=None), OK), (dict(m=0, accumulate=1, dy=None), OK),
])
def test_act_backward(lib, changes, want):
    assert call(lib.fp4_act_backward, BACK, **changes) == want


def test_act_backward_workspace(lib):
    size = lib.fp4_act_backward_workspace
    assert size(0, 64) == size(5, 0) == size(8, 256) == 0
    assert 0 < size(1 << 40, 32) <= 512 * 32 * 4 and size(8192, 14336) % (4 * 14336) == 0
    assert size(-1, 64) == size(1, 33) == size((1 << 40) + 1, 32) == size(1, (1 << 28) + 32) == -1


def test_capacity(lib):
    rows = lib.fp4_expert_capacity
    assert rows(0, 1, 1, 1) == rows(0, 2, 8, 32) == 0 and rows(5, 3, 8, 1) == 15
    assert rows(1, 2, 8, 32) == 256 and rows(8192, 8, 64, 32) == 65536 + 2048 and rows(3, 1, 1024, 256) == 768
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0), (1, 1, 1, 2), (1, 1, 1, 33), (1, 1, 1, 288),
                (1 << 31, 1, 1, 1), (1 << 40, 1 << 40, 1, 1)):
        assert rows(*bad) == -1, bad
    assert rows(1 << 30, 1, 1024, 256) <= (1 << 30) + (1 << 18)


def test_sort_workspace(lib):
    size = lib.fp4_expert_sort_workspace
    assert size(0, 1, 1) == size(64, 8, 1024) == 0 and size(1 << 17, 8, 64) > 0
    assert size(-1, 1, 1) == size(1, 1, 0) == size(1 << 31, 1, 1) == -1


SORT = dict(t=4, k=2, e=8, ids=P, id_bytes=4, align=32, capacity=512, offsets=P, slots=P, rows=P, ws=None, size=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(id_bytes=2), EINVAL), *each(("ids", "offsets", "slots", "rows"), None, EINVAL),
    (dict(t=1 << 17, k=8, capacity=1 << 21, size=1 << 30), EINVAL),
    (dict(t=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(e=0), ESHAPE), (dict(e=1025), ESHAPE), (dict(align=16), ESHAPE),
    (dict(capacity=255), ESHAPE), (dict(capacity=1 << 31), ESHAPE), (dict(t=1 << 17, k=8, capacity=1 << 21), ESHAPE),
    (dict(ids=P + 2), EALIGN), (dict(id_bytes=8, ids=P + 4), EALIGN), (dict(offsets=P + 2), EALIGN), (dict(slots=P + 2), EALIGN),
    (dict(rows=P + 2), EALIGN),
])
def test_sort(lib, changes, want):
    assert call(lib.fp4_expert_sort, SORT, **changes) == want


GATHER = dict(t=4, k=2, d=64, rows=512, x=P, ldx=64, slots=P, xs=P, fmt=0, codes=P, scales=P, ws=None, size=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(fmt=2), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(x=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(t=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(d=48), ESHAPE), (dict(ldx=56), ESHAPE), (dict(rows=-1), ESHAPE), (dict(rows=1 << 31), ESHAPE),
    (dict(t=1 << 31), ESHAPE), (dict(d=1 << 31, ldx=1 << 31), ESHAPE),
    (dict(x=P + 8), EALIGN), (dict(xs=P + 8), EALIGN), (dict(codes=P + 8), EALIGN), (dict(ldx=68), EALIGN), (dict(slots=P + 2), EALIGN), (dict(ws=P + 2), EALIGN),
    (dict(t=1 << 16, d=4096, ldx=4096, rows=1 << 17), ESHAPE), (dict(t=1 << 16, d=4096, ldx=4096, rows=1 << 17, size=1 << 20), EINVAL),
    (dict(rows=0, x=None, slots=None), OK), (dict(d=0, x=None), OK), (dict(xs=None, codes=None, scales=None), OK),
])
def test_gather(lib, changes, want):
    assert call(lib.fp4_expert_gather, GATHER, **changes) == want


COMBINE = dict(t=4, k=2, d=64, rows=8, z=P, zt=0, ldz=64, where=P, weights=P, res=P, ldr=64, out=P, ldo=64, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(zt=2), EINVAL), (dict(z=None), EINVAL), (dict(where=None), EINVAL), (dict(out=None), EINVAL),
    (dict(t=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(d=40), ESHAPE), (dict(rows=-1), ESHAPE), (dict(ldz=56), ESHAPE), (dict(ldr=56), ESHAPE),
    (dict(ldo=56), ESHAPE), (dict(t=1 << 30), ESHAPE), (dict(rows=1 << 31), ESHAPE),
    (dict(z=P + 8), EALIGN), (dict(res=P + 8), EALIGN), (dict(out=P + 8), EALIGN), (dict(ldz=68), EALIGN), (dict(zt=1, ldz=66), EALIGN),
    (dict(ldr=68), EALIGN), (dict(ldo=68), EALIGN), (dict(where=P + 2), EALIGN), (dict(weights=P + 2), EALIGN),
    (dict(t=0, z=None, where=None, out=None), OK), (dict(d=0, z=None, out=None), OK),
])
def test_combine(lib, changes, want):
    assert call(lib.fp4_expert_combine, COMBINE, **changes) == want


CBACK = dict(t=4, k=2, d=64, rows=8, dy=P, dyt=1, lddy=64, z=P, zt=0, ldz=64, slots=P, where=P, weights=P, dz=P, dw=P, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(dyt=2), EINVAL), (dict(zt=2), EINVAL), *each(("dy", "z", "slots", "where", "weights", "dz", "dw"), None, EINVAL),
    (dict(t=-1), ESHAPE), (dict(k=0), ESHAPE), (dict(d=40), ESHAPE), (dict(lddy=56), ESHAPE), (dict(ldz=56), ESHAPE), (dict(rows=-1), ESHAPE),
    *each(("dy", "z", "dz"), P + 8, EALIGN), *each(("slots", "where", "weights", "dw"), P + 2, EALIGN), (dict(lddy=66), EALIGN),
    (dict(ldz=68), EALIGN), (dict(t=0, rows=0, dy=None, z=None, dz=None), OK),
])
def test_combine_backward(lib, changes, want):
    assert call(lib.fp4_expert_combine_backward, CBACK, **changes) == want


EXP = dict(e=4, rows=40, n=64, k=96, offsets=P, ac=P, asc=P, bc=P, bsc=P, a2=None, a2s=None, b2=None, b2s=None, c=P, ct=1, ldc=64, stream=None)
NO_PAIR = dict(a2=P, a2s=P, b2=P, b2s=P)


@pytest.mark.parametrize("changes,want", [
    (dict(ct=2), EINVAL), *each(("offsets", "ac", "asc", "bc", "bsc", "c"), None, EINVAL),
    *((NO_PAIR | {n: None}, EINVAL) for n in NO_PAIR),
    (dict(e=0), ESHAPE), (dict(e=1025), ESHAPE), (dict(rows=-1), ESHAPE), (dict(rows=(1 << 30) + 1), ESHAPE), (dict(n=40), ESHAPE),
    (dict(k=40), ESHAPE), (dict(k=1 << 24), ESHAPE), (dict(ldc=56), ESHAPE), (dict(n=1 << 31, ldc=1 << 31), ESHAPE),
    *each(("ac", "asc", "bc", "bsc", "c"), P + 8, EALIGN), *((NO_PAIR | {n: P + 8}, EALIGN) for n in NO_PAIR), (dict(offsets=P + 2), EALIGN),
    (dict(ldc=66), EALIGN), (dict(ct=0, ldc=68), EALIGN),
    (dict(rows=0, offsets=None, c=None), OK), (dict(n=0, c=None), OK),
])
def test_gemm_experts(lib, changes, want):
    assert call(lib.fp4_gemm_experts, EXP, **changes) == want


WGRAD = dict(e=4, tokens=512, m=64, n=96, offsets=P, ac=P, asc=P, bc=P, bsc=P, c=P, ct=1, accumulate=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(ct=2), EINVAL), (dict(accumulate=2), EINVAL), (dict(ct=0, accumulate=1), EINVAL),
    *each(("offsets", "ac", "asc", "bc", "bsc", "c"), None, EINVAL),
    (dict(e=0), ESHAPE), (dict(tokens=-256), ESHAPE), (dict(tokens=288), ESHAPE), (dict(tokens=1 << 24), ESHAPE), (dict(m=40), ESHAPE),
    (dict(n=-32), ESHAPE), (dict(m=1 << 40), ESHAPE), *each(("ac", "asc", "bc", "bsc", "c"), P + 8, EALIGN), (dict(offsets=P + 2), EALIGN),
    (dict(m=0, c=None), OK), (dict(n=0, ac=None), OK),
])
def test_gemm_experts_wgrad(lib, changes, want):
    assert call(lib.fp4_gemm_experts_wgrad, WGRAD, **changes) == want


SWIGLU = dict(e=4, rows=64, f=64, d=96, offsets=P, xc=P, xs=P, wc=P, ws=P, a=P, b=P, hc=P, hs=P, htc=P, hts=P, signs=0, stream=None)


@pytest.mark.parametrize("changes,want", [
    (dict(htc=None), EINVAL), (dict(hts=None), EINVAL), *each(("offsets", "xc", "xs", "wc", "ws", "a", "b", "hc", "hs"), None, EINVAL),
    (dict(e=0), ESHAPE), (dict(rows=40), ESHAPE), (dict(f=40), ESHAPE), (dict(d=40), ESHAPE), (dict(d=1 << 24), ESHAPE), (dict(rows=-32), ESHAPE),
    *each(("xc", "xs", "wc", "ws", "a", "b", "hc", "htc"), P + 8, EALIGN), (dict(offsets=P + 2), EALIGN),
    (dict(rows=0, offsets=None, a=None), OK), (dict(f=0, a=None), OK),
])
def test_swiglu_producer_experts(lib, changes, want):
    assert call(lib.fp4_swiglu_producer_experts, SWIGLU, **changes) == want


MV = dict(e=4, rows=9, n=5, k=64, offsets=P, x=P, ldx=64, xs=None, codes=P, scales=P, c=P, ldc=5, stream=None)


@pytest.mark.parametrize("changes,want", [
    *each(("offsets", "x", "codes", "scales", "c"), None, EINVAL),
    (dict(e=0), ESHAPE), (dict(rows=-1), ESHAPE), (dict(rows=65537), ESHAPE), (dict(n=-1), ESHAPE), (dict(k=48), ESHAPE), (dict(ldx=56), ESHAPE),
    (dict(ldc=4), ESHAPE), (dict(xs=P, ldx=72), ESHAPE), (dict(x=P + 8), EALIGN), (dict(codes=P + 8), EALIGN), (dict(ldx=68), EALIGN),
    (dict(c=P + 2), EALIGN), (dict(offsets=P + 2), EALIGN), (dict(rows=0, x=None, c=None), OK), (dict(n=0, c=None), OK),
])
def test_matvec_experts(lib, changes, want):
    assert call(lib.fp4_matvec_experts, MV, **changes) == want


SMV = dict(e=4, rows=9, f=5, d=64, offsets=P, x=P, ldx=64, xs=None, codes=P, scales=P, h=P, stream=None)


@pytest.mark.parametrize("changes,want", [
    *each(("offsets", "x", "codes", "scales", "h"), None, EINVAL), (dict(rows=65537), ESHAPE), (dict(xs=P, ldx=72), ESHAPE),
    (dict(h=ODD), EALIGN), (dict(offsets=P + 2), EALIGN), (dict(rows=0, h=None), OK),
])
def test_swiglu_matvec_experts(lib, changes, want):
    assert call(lib.fp4_swiglu_matvec_experts, SMV, **changes) == want


def test_binding_refuses_host_tensors_by_name():
    import precision_mxfp4_producers_amd as mx
    u8, b16, i32 = torch.zeros((32, 32), dtype=torch.uint8), torch.zeros((32, 32)).bfloat16(), torch.zeros(5, dtype=torch.int32)
    calls = [(mx.fp4_gemm_act, (u8, u8, u8, u8), "a_codes"), (mx.fp4_matvec_act, (b16, u8, u8), "x"), (mx.fp4_act_backward, (b16, b16, 1), "dy"),
             (mx.fp4_expert_sort, (i32, 4), "ids"), (mx.fp4_expert_gather, (b16, i32, 1), "x"), (mx.fp4_expert_combine, (b16, i32), "z"),
             (mx.fp4_expert_combine_backward, (b16, b16, i32, i32, b16), "dy"), (mx.fp4_gemm_experts, (i32, u8, u8, u8, u8), "a_codes"),
             (mx.fp4_gemm_experts_wgrad, (i32, u8, u8, u8, u8), "a_codes"), (mx.fp4_swiglu_producer_experts, (i32, u8, u8, u8, u8), "x_codes"),
             (mx.fp4_matvec_experts, (i32, b16, u8, u8), "x"), (mx.fp4_swiglu_matvec_experts, (i32, b16, u8, u8), "x")]
    for fn, args, name in calls:
        with pytest.raises(mx.Fp4Error, match=f"^{name} must be a CUDA"):
            fn(*args)
