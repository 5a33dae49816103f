"""The norm with the residual's addition on the GPU, its outputs in 8 bits and its gradient,
against the float64 reference (oracle/layer_oracle.py).

Tolerances. Inside, every value is fp32: a row's sum of squares takes at most 32 sequential
additions in a thread (rows read twice: 64) and 22 across threads, 2^-24 of the sum each, halved by the root; the
root, the quotient and two products add 2^-24 each: below 2^-18 of y in all. The rounding at
the end adds half a step, 2^-8 (bf16) or 2^-24 (fp32). The gradient's two terms carry that
error each, the mean that of its own terms' sizes. Sums h and entries of 8 bits are IEEE
fp32 arithmetic of their definition: equal bit for bit. Weight gradients are sums of
T products, each off by 2^-18, in at most 2^6 sequential additions: 2^-17 of the summed sizes."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float32]
# every count of threads a row, the ends of their ranges, widths that end inside 16 bytes, rows read twice
WIDTHS = [1, 3, 8, 64, 257, 512, 513, 1000, 1001, 2048, 4096, 4099, 8200, 14336, 16385, 33000]


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(T, d, dtype, seed=0, pad=0):
    """x, residual, weight, g_y, g_h; views into rows of d + pad elements."""
    g = torch.Generator().manual_seed(seed)
    loud = 1 + 20 * (torch.rand(d, generator=g) < 0.02)

    def rows(scale):
        t = torch.zeros(T, d + pad, dtype=dtype)
        t[:, :d] = (torch.randn(T, d, generator=g) * scale).to(dtype)
        return t.cuda()[:, :d]

    return rows(1.0), rows(loud), (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda(), rows(0.3), rows(0.3)


def check_y(y, h, w, eps, dtype):
    ref = lo.norm(np64(h), np64(w), eps)
    bound = (HALF[dtype] + 2.0 ** -18) * np.abs(ref) + 1e-37
    assert (np.abs(np64(y) - ref) <= bound).all()


def check_eight(kind, y, scale, h, w, eps):
    """Entries from the definition in IEEE fp32 (torch on the CPU), the scale against 64 bits."""
    n = h.cpu().float() * (1.0 if w is None else w.cpu().float())
    top = torch.tensor(127.0 if kind == "int8" else 448.0)
    s = n.abs().amax(1, keepdim=True) / top
    q = torch.where(s > 0, n / s, torch.zeros(())).clamp(-top, top)
    if kind == "int8":
        assert y.dtype == torch.int8 and torch.equal(y.cpu(), q.round().to(torch.int8))
    else:
        assert y.dtype == torch.float8_e4m3fn
        assert torch.equal(y.cpu().view(torch.uint8), q.to(torch.float8_e4m3fn).view(torch.uint8))
    h64 = np64(h)
    ref = s[:, 0].double().numpy() / np.sqrt((h64 ** 2).mean(1) + eps)
    assert (np.abs(np64(scale) - ref) <= 2.0 ** -18 * ref).all()


def check_gradient(got, h, w, g_y, g_h, eps, dtype):
    h64, w64, gy, gh = np64(h), np64(w), np64(g_y), np64(g_h)
    rx, rw = lo.norm_backward(h64, w64, gy, gh, eps)
    r = 1 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + eps)
    u = np.abs(gy if w64 is None else gy * w64)
    xh = np.abs(h64) * r
    size = r * (u + xh * (u * xh).mean(1, keepdims=True)) + (0 if gh is None else np.abs(gh))
    assert got["x"].dtype == dtype
    assert (np.abs(np64(got["x"]) - rx) <= HALF[dtype] * np.abs(rx) + 2.0 ** -17 * size + 1e-37).all()
    if w is None:
        assert got["weight"] is None
    else:
        assert (np.abs(np64(got["weight"]) - rw) <= 2.0 ** -17 * (np.abs(gy) * xh).sum(0) + 1e-37).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("d", WIDTHS)
def test_every_width(d, T, dtype):
    import activation_sparse_ffn_amd as sffn
    x, r, w, gy, gh = make(T, d, dtype, seed=d + T)
    y, h = sffn.add_rms_norm(x, r, w, eps=1e-5)
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    check_y(y, h, w, 1e-5, dtype)
    for kind in ("int8", "e4m3"):
        q, scale, h2 = sffn.add_rms_norm(x, r, w, eps=1e-5, quant=kind)
        assert torch.equal(h2, h)
        check_eight(kind, q, scale, h, w, 1e-5)
    check_gradient(sffn.add_rms_norm_backward(h, gy, w, g_h=gh, eps=1e-5), h, w, gy, gh, 1e-5, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [100, 1001, 4096, 20000])
def test_without_residual_weight_or_second_gradient(d, dtype):
    import activation_sparse_ffn_amd as sffn
    x, _, w, gy, _ = make(7, d, dtype, seed=d)
    for weight in (w, None):
        y, h = sffn.add_rms_norm(x, weight=weight)
        assert h is x
        check_y(y, x, weight, 1e-6, dtype)
        check_eight("int8", *sffn.add_rms_norm(x, None, weight, quant="int8")[:2], x, weight, 1e-6)
        check_gradient(sffn.add_rms_norm_backward(x, gy, weight), x, weight, gy, None, 1e-6, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,pad", [(64, 1), (1000, 8), (4096, 3), (4097, 2), (20001, 5)])
def test_strides_and_what_lies_between_rows(d, pad, dtype):
    """Rows of any stride and alignment; what lies between them is neither read nor written."""
    import activation_sparse_ffn_amd as sffn
    x, r, w, gy, gh = make(6, d, dtype, seed=d, pad=pad)
    for t in (x, r, gy, gh):
        t._base[:, d:] = float("nan")
    big = torch.full((6, d + pad), 7.0, dtype=dtype, device="cuda")
    bigh = torch.full((6, d + pad), 7.0, dtype=dtype, device="cuda")
    y, h = sffn.add_rms_norm(x, r, w, y_out=big[:, :d], h_out=bigh[:, :d])
    assert (big[:, d:] == 7).all() and (bigh[:, d:] == 7).all()
    check_y(y, h, w, 1e-6, dtype)
    small = torch.full((6, d + pad), 7, dtype=torch.int8, device="cuda")
    q, scale, _ = sffn.add_rms_norm(x, r, w, quant="int8", y_out=small[:, :d])
    assert (small[:, d:] == 7).all()
    check_eight("int8", q, scale, h, w, 1e-6)
    check_gradient(sffn.add_rms_norm_backward(h, gy, w, g_h=gh), h, w, gy, gh, 1e-6, dtype)


@pytest.mark.parametrize("d", [300, 4096, 40000])
def test_outputs_in_place(d):
    import activation_sparse_ffn_amd as sffn
    x, r, w, _, _ = make(9, d, torch.bfloat16, seed=3)
    y, h = sffn.add_rms_norm(x, r, w)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        to_y, to_h = (b, a) if swap else (a, b)
        y2, h2 = sffn.add_rms_norm(a, b, w, y_out=to_y, h_out=to_h)
        assert y2 is to_y and h2 is to_h and torch.equal(y2, y) and torch.equal(h2, h)


@pytest.mark.parametrize("d", [100, 4096, 40000])
def test_rows_of_zeros_and_rows_that_are_not_finite(d):
    import activation_sparse_ffn_amd as sffn
    x, _, w, _, _ = make(5, d, torch.float32, seed=1)
    x[1] = 0
    x[2, d // 2] = float("nan")
    x[3, d - 1] = float("-inf")
    y, _ = sffn.add_rms_norm(x, None, w)
    assert (y[1] == 0).all() and y[2].isnan().all() and y[3, d - 1].isnan() and (y[3, :d - 1] == 0).all()
    check_y(y[[0, 4]], x[[0, 4]], w, 1e-6, torch.float32)
    for kind in ("int8", "e4m3"):
        q, s, _ = sffn.add_rms_norm(x, None, w, quant=kind)
        assert s[1] == 0 and (q[1].float() == 0).all() and s[2].isnan() and s[3].isnan()
        check_eight(kind, q[[0, 4]], s[[0, 4]], x[[0, 4]], w, 1e-6)


def test_entries_of_the_smallest_numbers():
    """A scale among fp32's denormal numbers is inexact: entries keep to their range."""
    import activation_sparse_ffn_amd as sffn
    x = torch.tensor([[3e-44, -1e-44, 0.0], [1e-38, -2e-39, 5e-45]], device="cuda")
    for kind in ("int8", "e4m3"):
        q, s, _ = sffn.add_rms_norm(x, quant=kind, eps=1e-20)
        assert (q.float().abs() <= (127 if kind == "int8" else 448)).all() and torch.isfinite(s).all()


def test_repeated_captured_and_on_another_stream():
    """Equal bits from call to call, from a captured graph's replays and from another stream."""
    import activation_sparse_ffn_amd as sffn
    x, r, w, gy, gh = make(2000, 1024, torch.bfloat16, seed=9)

    def call():
        y, h = sffn.add_rms_norm(x, r, w)
        q, s, _ = sffn.add_rms_norm(x, r, w, quant="e4m3")
        g = sffn.add_rms_norm_backward(h, gy, w, g_h=gh)
        return [y, h, q.view(torch.uint8), s, g["x"], g["weight"]]

    first = call()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = call()
    torch.cuda.current_stream().wait_stream(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = call()
    for _ in range(3):
        for t in third:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, third):
            assert torch.equal(a, b) and torch.equal(a, c)
        x.add_(0)


def test_no_rows():
    import activation_sparse_ffn_amd as sffn
    x = torch.empty(0, 100, device="cuda")
    w = torch.ones(100, device="cuda")
    y, h = sffn.add_rms_norm(x, x, w)
    assert y.shape == h.shape == (0, 100)
    g = sffn.add_rms_norm_backward(x, x, w)
    assert g["x"].shape == (0, 100) and (g["weight"] == 0).all()


def test_more_rows_than_a_pass_takes():
    """Workgroups of the gradient take several rows each, and the last ones none."""
    import activation_sparse_ffn_amd as sffn
    for T, d, dtype in ((5000, 192, torch.bfloat16), (4111, 777, torch.float32), (1025, 1000, torch.bfloat16)):
        x, r, w, gy, gh = make(T, d, dtype, seed=T)
        check_gradient(sffn.add_rms_norm_backward(r, gy, w, g_h=gh), r, w, gy, gh, 1e-6, dtype)
