"""Head norms with rotary positions on the GPU, forward and backward, against
the float64 reference (oracle/attention_oracle.py).

Tolerances. Inside, every value is fp32: the norm's sum of D <= 512 squares, its
root and three products put at most about 2^-19 of relative error on a turned
element's terms, |n_a c| + |n_b s| <= 2 max|n| of the head's row; the one
rounding at the end adds 2^-9 (bf16) or 2^-24 (fp32) of the result. The
gradient's terms are sums of three such products. So

  |y - ref| <= eps |ref| + 2^-18 max|ref row| (forward; * 4 backward)

with the row's largest element for the terms' size. Weight gradients are fp32
sums of T H products, each off by 2^-19 of its size at most, added in at most
2^11 sequential steps: |g - ref| <= 2^-13 of the root of the summed squares."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(y, ref, dtype, factor=1.0):
    y = np64(y)
    assert y.shape == ref.shape
    bound = EPS[dtype] * np.abs(ref) + factor * 2.0 ** -18 * np.abs(ref).max(-1, keepdims=True) + 1e-30
    worst = (np.abs(y - ref) / bound).max() if ref.size else 0.0
    assert worst <= 1, f"{worst:.2f} times the bound"


def make(T, H, K, D, rot, dtype, seed, packed=False, weights=True, max_pos=4096):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, H + 2 * K, D, generator=g).to(dtype).cuda()
    q, k = qkv[:, :H], qkv[:, H:H + K]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() if weights else None for _ in range(2)]
    pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32).cuda()
    gq, gk = (torch.randn(T, n, D, generator=g).to(dtype).cuda() for n in (H, K))
    return q, k, w[0], w[1], pos, gq, gk


def table(rot, max_pos=4096, **kw):
    import activation_sparse_ffn_amd as sffn
    return sffn.rope_table(max_pos, rot, **kw) if rot else None


def check(T, H, K, D, rot, dtype, layout, norm, seed=0, packed=False, weights=True):
    import activation_sparse_ffn_amd as sffn
    weights = weights and norm
    q, k, wq, wk, pos, gq, gk = make(T, H, K, D, rot, dtype, seed, packed, weights)
    t = table(rot)
    kw = dict(norm=norm, eps=1e-5, layout=layout)
    yq, yk = sffn.qk_norm_rope(q, k, pos, t, wq, wk, **kw)
    g = sffn.qk_norm_rope_backward(q, k, gq, gk, pos, t, wq, wk, **kw)
    torch.cuda.synchronize()
    p, tt = pos.cpu().numpy(), None if t is None else t.cpu().numpy()
    for n, x, w, y, gy in (("q", q, wq, yq, gq), ("k", k, wk, yk, gk)):
        close(y, ao.norm_rope(np64(x), p, tt, np64(w), **kw), dtype)
        rx, rw = ao.norm_rope_backward(np64(x), np64(gy), p, tt, np64(w), **kw)
        close(g[n], rx, dtype, 4)
        if weights:
            gn = np64(gy) if t is None else ao.rotate(np64(gy), p, tt, layout, back=True)
            size = np.sqrt(((gn * ao.norm_rope(np64(x), p, None, None, eps=1e-5)) ** 2).sum((0, 1))).max()
            assert (np.abs(np64(g[n + "_weight"]) - rw) <= 2.0 ** -13 * size).all()
        else:
            assert g[n + "_weight"] is None


# the 16-byte kernels: every lane group, both layouts, part of the head, tokens from one on
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,K,D,rot,layout,norm", [
    (1, 32, 8, 128, 128, "half", True),
    (1, 1, 1, 64, 64, "interleaved", True),
    (7, 4, 4, 64, 32, "half", True),
    (33, 7, 1, 80, 32, "half", True),
    (33, 7, 1, 80, 40, "interleaved", True),
    (65, 12, 3, 96, 96, "half", False),
    (65, 12, 3, 96, 24, "interleaved", False),
    (300, 28, 4, 128, 64, "interleaved", True),
    (19, 8, 2, 256, 256, "half", True),
    (19, 8, 2, 256, 240, "half", True),
    (5, 3, 1, 512, 512, "half", True),
    (5, 2, 2, 8, 8, "interleaved", True),
    (1500, 32, 8, 128, 128, "half", True),
])
def test_wide(T, H, K, D, rot, layout, norm, dtype):
    check(T, H, K, D, rot, dtype, layout, norm, seed=T + D)


# the element-wise kernel: odd head sizes, rotated parts that do not fill eights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,K,D,rot,layout,norm", [
    (1, 1, 1, 2, 2, "half", True),
    (1, 2, 1, 1, 0, "half", True),
    (9, 3, 1, 65, 64, "half", True),
    (9, 3, 1, 65, 64, "interleaved", True),
    (17, 5, 5, 100, 50, "half", True),
    (17, 5, 5, 100, 50, "interleaved", False),
    (40, 2, 1, 128, 72, "half", True),
    (3, 2, 2, 511, 510, "half", True),
    (700, 9, 3, 36, 36, "half", True),
])
def test_any_size(T, H, K, D, rot, layout, norm, dtype):
    check(T, H, K, D, rot, dtype, layout, norm, seed=T + D)


@pytest.mark.parametrize("D", [128, 72])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_without_weights_and_rotation_alone(D, layout):
    check(13, 4, 2, D, 64, torch.bfloat16, layout, True, weights=False)
    check(13, 4, 2, D, 64, torch.float32, layout, False)
    check(13, 4, 2, D, 0, torch.float32, layout, True)


@pytest.mark.parametrize("D", [128, 100])
def test_views_of_a_packed_projection(D):
    check(50, 6, 2, D, 64, torch.bfloat16, "half", True, packed=True)


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 32), (90, 60)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_head_major_outputs(D, rot, layout):
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, _, _ = make(37, 5, 2, D, rot, torch.bfloat16, 3)
    t = table(rot)
    yq, yk = sffn.qk_norm_rope(q, k, pos, t, wq, wk, layout=layout)
    heads = torch.empty(5, 37, D, dtype=q.dtype, device="cuda").transpose(0, 1)
    oq, _ = sffn.qk_norm_rope(q, k, pos, t, wq, wk, layout=layout, q_out=heads)
    assert oq is heads and torch.equal(heads, yq)
    q2, k2 = q.clone(), k.clone()
    sffn.qk_norm_rope(q2, k2, pos, t, wq, wk, layout=layout, q_out=q2, k_out=k2)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)


def test_q_alone_and_no_tokens():
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, gq, _ = make(6, 4, 2, 64, 64, torch.bfloat16, 4)
    t = table(64)
    both, _ = sffn.qk_norm_rope(q, k, pos, t, wq, wk)
    alone, none = sffn.qk_norm_rope(q, None, pos, t, wq)
    assert none is None and torch.equal(both, alone)
    g = sffn.qk_norm_rope_backward(q, None, gq, None, pos, t, wq)
    assert g["k"] is None and g["k_weight"] is None and g["q_weight"] is not None
    e = q[:0]
    y, z = sffn.qk_norm_rope(e, k[:0], pos[:0], t, wq, wk)
    assert y.shape == e.shape and z.shape == (0, 2, 64)
    g = sffn.qk_norm_rope_backward(e, k[:0], gq[:0], k[:0], pos[:0], t, wq, wk)
    torch.cuda.synchronize()
    assert (g["q_weight"] == 0).all() and (g["k_weight"] == 0).all()


@pytest.mark.parametrize("D", [128, 90])
def test_positions_outside_the_table_are_nan(D):
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, _, _ = make(5, 3, 1, D, 64, torch.float32, 5)
    t = table(64)
    good, _ = sffn.qk_norm_rope(q, k, pos, t, wq, wk)
    bad = pos.clone()
    bad[1], bad[3] = -1, t.shape[0]
    y, z = sffn.qk_norm_rope(q, k, bad, t, wq, wk)
    for i in range(5):
        if i in (1, 3):
            assert y[i].isnan().all() and z[i].isnan().all()
        else:
            assert torch.equal(y[i], good[i])


@pytest.mark.parametrize("D", [128, 90])
def test_zeros_infinities_and_nan_stay_in_their_head(D):
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, _, _ = make(4, 3, 1, D, 64, torch.bfloat16, 6)
    t = table(64)
    good, _ = sffn.qk_norm_rope(q, k, pos, t, wq, wk)
    q[0, 0] = 0
    q[1, 1, 5] = float("inf")
    q[2, 2, 7] = float("nan")
    y, _ = sffn.qk_norm_rope(q, k, pos, t, wq, wk)
    assert (y[0, 0] == 0).all() and y[1, 1].isnan().any() and y[2, 2].isnan().all()
    same = torch.ones(4, 3, dtype=torch.bool)
    same[0, 0] = same[1, 1] = same[2, 2] = False
    assert torch.equal(y[same], good[same])


@pytest.mark.parametrize("D", [64, 90])
def test_gradient_against_differences_of_the_forward(D):
    """Central differences of the fp32 forward itself, h = 2^-6: the third
    derivative's h^2 / 6 share is under 2^-12 of the row's size here, and the
    fp32 sums' rounding over 2 h about 2^-24 D 2^5 ~ 2^-12."""
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, gq, gk = make(2, 1, 1, D, 32, torch.float32, 7)
    t = table(32)
    g = sffn.qk_norm_rope_backward(q, k, gq, gk, pos, t, wq, wk, eps=1e-5)
    h = 2.0 ** -6
    for d in range(0, D, 7):
        moved = []
        for s in (h, -h):
            x = q.clone()
            x[1, 0, d] += s
            y, _ = sffn.qk_norm_rope(x, k, pos, t, wq, wk, eps=1e-5)
            moved.append((y.double() * gq.double()).sum().item())
        assert abs((moved[0] - moved[1]) / (2 * h) - g["q"][1, 0, d].item()) < 2e-3


def test_same_bits_every_time_and_on_another_stream():
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, gq, gk = make(900, 8, 2, 128, 128, torch.bfloat16, 8)
    t = table(128)
    first = sffn.qk_norm_rope_backward(q, k, gq, gk, pos, t, wq, wk)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = sffn.qk_norm_rope_backward(q, k, gq, gk, pos, t, wq, wk)
    s.synchronize()
    assert all(torch.equal(first[n], again[n]) for n in first)


def test_scaled_tables():
    """linear: position p of a table for a context f times longer is position p /
    f of the trained one; ntk and by_parts keep the fastest pair and slow the
    slowest by f."""
    import activation_sparse_ffn_amd as sffn
    plain = sffn.rope_table(64, 32)
    linear = sffn.rope_table(256, 32, scaling="linear", factor=4.0)
    assert torch.allclose(linear[::4], plain, atol=1e-6)
    ntk = sffn.rope_table(256, 32, scaling="ntk", factor=4.0)
    assert torch.allclose(ntk[:64, [0, 16]], plain[:, [0, 16]], atol=1e-6)
    assert torch.allclose(ntk[::4, [15, 31]], plain[:, [15, 31]], atol=1e-6)
    parts = sffn.rope_table(256, 32, scaling="by_parts", factor=4.0, original_max_pos=1024)
    a = 1 + 0.1 * np.log(4.0)
    assert torch.allclose(parts[:64, [0, 16]], a * plain[:, [0, 16]], atol=1e-5)
    assert torch.allclose(parts[::4, [15, 31]], a * plain[:, [15, 31]], atol=1e-5)


def test_refusals():
    import activation_sparse_ffn_amd as sffn
    q, k, wq, wk, pos, gq, gk = make(4, 4, 2, 64, 64, torch.bfloat16, 9)
    t = table(64)
    for bad in (lambda: sffn.qk_norm_rope(q, k, pos, t, wq, wk, layout="other"),
                lambda: sffn.qk_norm_rope(q, k, pos, t, wq, wk, norm=False),
                lambda: sffn.qk_norm_rope(q, k, pos.long(), t),
                lambda: sffn.qk_norm_rope(q, k, pos[:3], t),
                lambda: sffn.qk_norm_rope(q, k, pos, t.double()),
                lambda: sffn.qk_norm_rope(q, k[:3], pos, t),
                lambda: sffn.qk_norm_rope(q, k.float(), pos, t),
                lambda: sffn.qk_norm_rope(q.half(), k.half(), pos, t),
                lambda: sffn.qk_norm_rope(q.cpu(), k, pos, t),
                lambda: sffn.qk_norm_rope(q[..., ::2], k[..., ::2], pos, t),
                lambda: sffn.qk_norm_rope(q, k, pos, t, wq.float(), wk),
                lambda: sffn.qk_norm_rope(q, k, pos, t, q_out=gq[:3])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sffn.qk_norm_rope(q, k, pos, table(66)),
                lambda: sffn.qk_norm_rope(q, k, pos, t, wq, wk, eps=0.0),
                lambda: sffn.qk_norm_rope(q, k, pos, t, q_out=gq[:1].expand(4, 4, 64))):
        with pytest.raises(sffn.SparseFFNError):
            bad()
