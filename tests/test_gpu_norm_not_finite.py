"""The norm's 8-bit outputs where a weight, or an entry times its weight, is not finite: the
row's scale says so. A scale is the largest |h w| over 127 or 448 times the row's factor, and
the largest of numbers among which is a NaN is NaN, so nothing is compared but NaN."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

# rows of one wave, of a workgroup, of several pieces a thread, read twice
WIDTHS = [5, 100, 4096, 4099, 16384, 40000]


def rows(d, dtype):
    g = torch.Generator().manual_seed(d)
    x, r = (torch.randn(6, d, generator=g).to(dtype).cuda() for _ in range(2))
    return x, r, (1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", WIDTHS)
def test_a_weight_that_is_not_finite(d, dtype, kind):
    import activation_sparse_ffn_amd as sffn
    x, r, w = rows(d, dtype)
    x[2], r[2] = 0, 0
    _, clean, h = sffn.add_rms_norm(x, r, w, quant=kind)
    assert torch.isfinite(clean).all()
    for bad in (float("nan"), float("inf"), float("-inf")):
        for at in (0, d // 2, d - 1):
            worse = w.clone()
            worse[at] = bad
            y, _ = sffn.add_rms_norm(x, r, worse)
            assert not torch.isfinite(y[:, at].float()).any()
            q, s, h2 = sffn.add_rms_norm(x, r, worse, quant=kind)
            assert s.isnan().all() and torch.equal(h2, h)
            assert (q.float() * s[:, None]).isnan().all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d", WIDTHS)
def test_a_product_beyond_fp32(d, kind):
    """One row's entry times its weight overflows; the other rows are as without it."""
    import activation_sparse_ffn_amd as sffn
    x, _, w = rows(d, torch.float32)
    w[d - 1] = 1e30
    x[:, d - 1] = 1e-30
    want, scale, _ = sffn.add_rms_norm(x, None, w, quant=kind)
    x[4, d - 1] = 1e15
    q, s, _ = sffn.add_rms_norm(x, None, w, quant=kind)
    others = [0, 1, 2, 3, 5]
    assert s[4].isnan() and torch.equal(s[others], scale[others])
    assert torch.equal(q[others].view(torch.uint8), want[others].view(torch.uint8))
