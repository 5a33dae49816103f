"""Pins of the float64 reference of the operators between a decoder layer's halves:
closed forms and central differences."""
import numpy as np
import pytest

from oracle import layer_oracle as lo


def test_norm_by_hand():
    h = np.array([[3.0, 4.0], [0.0, 0.0], [-1.0, 1.0]])
    y = lo.norm(h, np.array([1.0, 2.0]), 1e-300)
    r = np.sqrt(12.5)
    assert np.allclose(y[0], [3 / r, 8 / r]) and (y[1] == 0).all() and np.allclose(y[2], [-1, 2])
    assert np.allclose(lo.norm(np.array([[2.0, 2.0]]), None, 5.0), [[2 / 3, 2 / 3]])


@pytest.mark.parametrize("weighted", [True, False])
def test_norm_gradient_by_differences(weighted):
    rng = np.random.default_rng(1)
    h, g_y, g_h = (rng.normal(size=(3, 5)) for _ in range(3))
    w = rng.normal(size=5) if weighted else None

    def loss(h, w):
        return (lo.norm(h, w, 1e-3) * g_y).sum() + (h * g_h).sum()

    g_x, g_w = lo.norm_backward(h, w, g_y, g_h, 1e-3)
    e = 1e-6
    for t, i in np.ndindex(3, 5):
        d = np.zeros((3, 5))
        d[t, i] = e
        assert np.isclose(g_x[t, i], (loss(h + d, w) - loss(h - d, w)) / (2 * e), rtol=1e-6, atol=1e-8)
    if weighted:
        for i in range(5):
            d = np.zeros(5)
            d[i] = e
            assert np.isclose(g_w[i], (loss(h, w + d) - loss(h, w - d)) / (2 * e), rtol=1e-6, atol=1e-8)
