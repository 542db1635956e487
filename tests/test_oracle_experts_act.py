"""The oracle of the expert and epilogue calls, against differences, brute force
and the statements of the order."""

import numpy as np
import pytest

from oracle import act as A
from oracle import experts as X


@pytest.mark.parametrize("act", range(5))
def test_slope_is_the_derivative(act):
    z = np.linspace(-9, 9, 2001) + 1e-3                    # off relu's corner
    h = 1e-5
    diff = (A.value(z + h, act) - A.value(z - h, act)) / (2 * h)
    # central differences: h^2 / 6 of a third derivative below 3, and 2^-53 |z| / h of the values
    assert np.abs(diff - A.slope(z, act)).max() < 1e-9


def test_values_at_known_points():
    assert A.value(0.0, A.GELU) == 0 and abs(A.value(1.0, A.GELU) - 0.8413447460685429) < 1e-15
    assert abs(A.value(1.0, A.SILU) - 0.7310585786300049) < 1e-15
    assert abs(A.value(1.0, A.GELU_TANH) - 0.8411919906082768) < 1e-15
    assert A.value(-50.0, A.RELU) == 0 and A.value(-3.5, A.NONE) == -3.5


@pytest.mark.parametrize("align", [1, 32, 256])
@pytest.mark.parametrize("t,k,e", [(0, 1, 1), (1, 1, 1), (7, 3, 5), (100, 2, 70)])
def test_sort_order(t, k, e, align):
    rng = np.random.default_rng(t + k + e)
    ids = rng.integers(-1, e + 1, (t, k))
    offsets, slots, where = X.sort(ids, e, align)
    assert (np.diff(offsets) >= 0).all() and (offsets % align == 0).all() and offsets[e] <= len(slots)
    for i in range(e):
        seg = slots[offsets[i]:offsets[i + 1]]
        real = seg[seg >= 0]
        assert (np.diff(real) > 0).all() and (ids.reshape(-1)[real] == i).all() and (seg[len(real):] == -1).all()
        assert len(seg) - len(real) < align
    assert sorted(slots[slots >= 0]) == [s for s in range(t * k) if 0 <= ids.reshape(-1)[s] < e]
    assert all(slots[r] == s for s, r in enumerate(where.reshape(-1)) if r >= 0)


def test_combine_and_its_gradients_by_differences():
    rng = np.random.default_rng(3)
    ids = np.array([[0, 2], [2, -1], [1, 0]])
    _, slots, where = X.sort(ids, 3, 1)
    z, w, dy = rng.normal(size=(len(slots), 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))

    def loss(z, w):
        return (X.combine(z, where, w)[0] * dy).sum()

    dz, dw, _ = X.combine_backward(dy, z, where, w)
    h = 1e-6
    for i in np.ndindex(z.shape):
        d = np.zeros_like(z)
        d[i] = h
        assert abs((loss(z + d, w) - loss(z - d, w)) / (2 * h) - dz[i]) < 1e-8
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(z, w + d) - loss(z, w - d)) / (2 * h) - dw[i]) < 1e-8
