"""Pins of the float64 reference of the attention-side operators: closed forms,
central differences and a separately written softmax."""
import numpy as np
import pytest

from oracle import attention_oracle as ao


def table(max_pos, rot, base=100.0):
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_length_and_relative_angles(layout):
    """The dot product of a turned q and a turned k depends on the difference of
    their positions alone, and elements beyond the table pass."""
    rng = np.random.default_rng(0)
    t = table(50, 6)
    q, k = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))

    def dot(a, b):
        return (ao.rotate(q, np.array([a]), t, layout) * ao.rotate(k, np.array([b]), t, layout)).sum()

    assert np.isclose(dot(3, 10), dot(20, 27), atol=1e-12)
    y = ao.rotate(q, np.array([7]), t, layout)
    assert np.isclose((y ** 2).sum(), (q ** 2).sum()) and (y[..., 6:] == q[..., 6:]).all()
    assert np.allclose(ao.rotate(y, np.array([7]), t, layout, back=True), q)


def test_layouts_by_hand():
    t = np.array([[0.0, 0.0, 1.0, 1.0]])      # cos 0, sin 1: (a, b) -> (-b, a)
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    pos = np.array([0])
    assert (ao.rotate(x, pos, t, "half") == [[[-3, -4, 1, 2]]]).all()
    assert (ao.rotate(x, pos, t, "interleaved") == [[[-2, 1, -4, 3]]]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_gradient_against_differences(layout, norm):
    rng = np.random.default_rng(1)
    x, g, w, t = rng.normal(size=(3, 2, 10)), rng.normal(size=(3, 2, 10)), rng.normal(size=10), table(9, 6)
    pos = np.array([0, 4, 8])
    kw = dict(norm=norm, eps=1e-3, layout=layout)

    def loss(x, w):
        return (ao.norm_rope(x, pos, t, w if norm else None, **kw) * g).sum()

    gx, gw = ao.norm_rope_backward(x, g, pos, t, w if norm else None, **kw)
    h = 1e-6
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - gx[i]) < 1e-7
    if norm:
        for i in range(10):
            d = np.zeros(10)
            d[i] = h
            assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - gw[i]) < 1e-7


def test_append_by_hand():
    c = ao.Cache(2, 1, 4, 2)
    c.append([1, 0], 0, np.array([[[127.0, -63.6]]], np.float32), np.array([[[0.0, 0.0]]], np.float32))
    assert c.k_scale[1, 0] == 1 and c.keys[1, 0, 0].tolist() == [127, -64]
    assert c.v_scale[1, 0] == 0 and (c.values[1, 0, 0] == 0).all()
    # twice the range: the held entries are rounded to even halves
    c.append([1, 0], 1, np.array([[[254.0, 5.0]]], np.float32), np.array([[[1.0, -1.0]]], np.float32))
    assert c.k_scale[1, 0] == 2
    assert c.keys[1, 0, :2].tolist() == [[64, -32], [127, 2]]
    # a smaller token keeps the scale; the fifth one opens page 0
    c.append([1, 0], 2, np.ones((3, 1, 2), np.float32), np.ones((3, 1, 2), np.float32))
    assert c.k_scale[1, 0] == 2 and c.keys[1, 0, 3].tolist() == [0, 0]      # 1 / 2 rounds to even
    assert c.k_scale[0, 0] == np.float32(1) / np.float32(127) and c.keys[0, 0, 0].tolist() == [127, 127]
    # NaN poisons a page, and a fresh use of it clears that
    c.append([0], 1, np.full((1, 1, 2), np.nan, np.float32), np.ones((1, 1, 2), np.float32))
    assert np.isnan(c.k_scale[0, 0]) and c.v_scale[0, 0] == np.float32(1) / np.float32(127)
    c.append([0], 0, np.ones((1, 1, 2), np.float32), np.ones((1, 1, 2), np.float32))
    assert c.k_scale[0, 0] == np.float32(1) / np.float32(127)


def test_read_is_close_to_what_was_stored():
    rng = np.random.default_rng(3)
    c = ao.Cache(5, 3, 16, 8)
    k, v = rng.normal(size=(40, 3, 8)).astype(np.float32), rng.normal(size=(40, 3, 8)).astype(np.float32)
    for a, b in ((0, 1), (1, 7), (7, 33), (33, 40)):
        c.append([4, 0, 2], a, k[a:b], v[a:b])
    k2, v2 = c.read([4, 0, 2], 0, 40)
    # one rounding, or one more each time the scale of a page grew: at most 3 in a page here
    assert np.abs(k2 - k).max() < 3 * np.abs(k).max() / 127 and np.abs(v2 - v).max() < 3 * np.abs(v).max() / 127


def test_attention_against_a_masked_softmax():
    rng = np.random.default_rng(4)
    n, H, K, D, L, window = 5, 4, 2, 8, 9, 3
    q, k, v = rng.normal(size=(n, H, D)), rng.normal(size=(L, K, D)), rng.normal(size=(L, K, D))
    out, lse, _, _ = ao.attend(q, k, v, L - n, 0.3, window)
    kk, vv = np.repeat(k, H // K, 1), np.repeat(v, H // K, 1)
    s = 0.3 * np.einsum("ihd,jhd->hij", q, kk)
    i, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
    s = np.where((j <= i) & (j > i - window), s, -np.inf)
    e = np.exp(s)
    assert np.allclose(lse.T, np.log(e.sum(-1)))
    assert np.allclose(out, np.einsum("hij,jhd->ihd", e / e.sum(-1, keepdims=True), vv))


def test_rows_without_keys():
    q = np.ones((3, 1, 4))
    out, lse, _, _ = ao.attend(q, np.ones((1, 1, 4)), np.ones((1, 1, 4)), -2, 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and (out[2] == 1).all()
