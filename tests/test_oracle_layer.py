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


def test_plan_by_hand():
    """Pages of 16. The first sequence gives its second page back and begins a new one, the
    second ends, the third takes what came back first, and one page is lacking."""
    table, free, n, lacking, lens, cu, pos, slots = lo.plan(
        [[5, 7, -1], [2, 9, -1], [-1, -1, -1]], [30, 17, 0], [16, 0, 0], [1, 0, 65], [1, -1, -1, -1, -1, -1, -1, -1, -1, -1],
        1, 16, 70)
    # onto the stack: 7, 2, 9 above 1; off it: 9 for the first sequence, 2, 7, 1 for the third
    assert table == [[5, 9, -1], [2, 9, -1], [2, 7, 1]] and n == 0 and lacking == 0
    assert lens == [17, 0, 65] and cu == [0, 1, 1, 66]
    assert pos[0] == 16 and slots[0] == 9 * 16 and pos[1:66] == list(range(65))
    assert slots[1] == 32 and slots[17] == 7 * 16 and slots[33] == 16 and slots[48] == 31
    assert slots[49:66] == [-1] * 17        # behind the table's three pages
    assert slots[66:] == [-1] * 4 and pos[66:] == [0] * 4
    short = lo.plan([[-1, -1]], [0], None, [20], [3, 0, 0, 0], 1, 16, 20)
    assert short[0] == [[3, -1]] and short[3] == 1 and short[7] == [48 + i for i in range(16)] + [-1] * 4
