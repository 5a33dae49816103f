"""What attention over the 4-bit cache keeps of a bf16 q, in heads of 128 and in sequences of up
to 128 rows: its own entries, not their products with the scale.

Rows of equal entries m = 1 + i / 128 over one key of entries 6: every product, and the sum of
D of them, is a multiple of 2^-7 below 2^13, exact in fp32. (Cut after a product with scale
log2 e, m leaves up to 2^-17.9 of itself, in every channel the same.) What rounds is the score
times the scale's rest, the subtraction of the reference (itself: zero or a step of it), the
logarithm of the sum, 0 within 2^-22, the product with ln 2 and its constant: five steps of
2^-24 of the result, and 2^-22."""
import numpy as np
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# rows of a sequence and key head: a tile of 16, two, row tiles of several sequences and of one;
# more than 128, in heads of 128
SIZES = [(seqs, G, D) for seqs, G in ((128, 1), (16, 8), (8, 16), (4, 32), (2, 64), (1, 128)) for D in (64, 128, 256)]


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("seqs,G,D", SIZES + [(1, 256, 128), (3, 256, 128)])
def test_q_is_kept_whole(seqs, G, D, sign):
    import activation_sparse_ffn_amd as sffn
    m = 1 + torch.arange(seqs * G, dtype=torch.float64) % 128 / 128
    q = m.view(seqs, G, 1).expand(seqs, G, D).bfloat16().contiguous().cuda()
    assert torch.equal(q[..., 0].double().flatten().cpu(), m)
    cache = sffn.KVCache4.empty(seqs, 1, D, 16)
    batch = sffn.CacheBatch(i32(np.arange(seqs)[:, None]), i32([1] * seqs), 1)
    k = torch.full((seqs, 1, D), 6.0, device="cuda")
    sffn.kv_cache_append(cache, batch, k, k)
    for scale in (sign * D ** -0.5, sign * 0.1, sign * 0.7):
        o, lse = sffn.cache_attention(cache, batch, q, scale=scale, return_lse=True)
        assert (o == 6).all()
        want = float(np.float32(scale)) * 6 * D * m
        off = (lse.flatten().double().cpu() - want).abs()
        assert (off <= 5 * 2.0 ** -24 * want.abs() + 2.0 ** -22).all(), (off / want.abs()).max().item()
