"""Pins of the reference of the 4-bit cache: its format by hand, its attention against a
softmax written apart."""
import numpy as np

from oracle import cache4_oracle as co


def test_format_by_hand():
    q = np.array([0.0, 0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.75, 2.5, 2.5000001, 3.5, 5.0, 5.0000001, 6.0, -0.75, -3.0])
    want = [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 10, 13]
    assert co.encode(q).tolist() == want
    assert co.decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    c = np.arange(16, dtype=np.uint8)
    assert co.pack(c).tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] and (co.unpack(co.pack(c)) == c).all()


def test_scales_by_hand():
    k = np.zeros((6, 64), np.float32)
    k[0, 0], k[0, 40] = 6.0, -6.1
    k[1, 3], k[1, 63] = 1.5, 3.0 * 2.0 ** -140
    k[2, 1] = np.inf
    k[3, 35] = np.nan
    k[4, 0] = np.finfo(np.float32).max
    codes, e = co.quantise_keys(k)
    assert e.tolist() == [[127, 128], [125, 0], [255, 127 - 127], [0, 255], [253, 0], [0, 0]]
    assert codes[0, 0] == 7 and codes[0, 40] == 8 + 5 and codes[1, 3] == 7 and codes[4, 0] == 6
    # the least power of two, whatever the number
    x = np.exp(np.random.default_rng(0).uniform(-80, 80, (500, 1))).astype(np.float32) * np.ones((1, 32), np.float32)
    _, e = co.quantise_keys(x)
    top, two = x[:, :1].astype(np.float64), 2.0 ** (e.astype(np.float64) - 127)
    assert (top <= 6 * two).all() and (top > 3 * two).all()
    v = np.array([[3.0, -1.5, 0.25, 0.0], [0, 0, 0, 0], [1, np.nan, 0, 0]], np.float32)
    codes, s = co.quantise_values(v)
    assert s[0] == 0.5 and s[1] == 0 and np.isnan(s[2]) and codes[0].tolist() == [7, 13, 1, 0] and not codes[1].any()


def test_attention_against_a_plain_softmax():
    rng = np.random.default_rng(2)
    q, codes = rng.normal(size=(3, 4, 64)), rng.integers(0, 16, (9, 2, 64)).astype(np.uint8)
    k, sv = rng.normal(size=(9, 2, 64)), rng.uniform(0.1, 1, (9, 2))
    out, lse, w, W, a, b = co.attend(q, k, codes, sv, 6, 0.3, 4)
    v = co.decode(codes) * sv[..., None]
    for i in range(3):
        for h in range(4):
            s = 0.3 * k[3 + i:7 + i, h // 2] @ q[i, h]
            p = np.exp(s) / np.exp(s).sum()
            assert np.allclose(out[i, h], p @ v[3 + i:7 + i, h // 2]) and np.isclose(lse[i, h], np.log(np.exp(s).sum()))
    assert (W >= w - 1e-12).all() and (b >= a).all() and (w >= np.abs(out) - 1e-12).all()
