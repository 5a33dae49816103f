"""Row tiles of the 4-bit cache's attention over thousands of keys, one sequence's (cut into
ranges of keys) and several sequences' (cut into shares), against the float64 reference.

The bounds are those of test_gpu_cache4.py but for the sums over the keys: a part of n keys
adds n / 64 times as many products as the weights have pieces, 2^-24 of the sizes summed each,
and no part has more keys than the sequence: 2^-24 of w for each piece of each 64 keys, and
as much for l."""
import numpy as np
import pytest
import torch

from tests.conftest import gpu_available
from tests.test_gpu_cache4 import BF, F32, Setup, queries, reference

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv,new,H,K,D,page,window", [
    ([12000], [34], 2, 1, 128, 64, 0), ([9000], [9], 16, 1, 64, 16, 0), ([7000], [33], 1, 1, 256, 128, 0),
    ([9000, 300, 6000], [20, 40, 3], 2, 1, 128, 64, 0), ([8000, 5000, 70], [17, 5, 40], 2, 1, 256, 32, 0),
    ([9000, 4000], [40, 35], 1, 1, 64, 64, 3500),
])
def test_rows_over_thousands_of_keys(kv, new, H, K, D, page, window, dtype):
    s = Setup(kv, K, D, page, 31)
    q = queries(sum(new), H, D, dtype, 32)
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new), q, window=window, return_lse=True)
    torch.cuda.synchronize()
    (out, rl, w, W, a, b), many = reference(s, q, new, D ** -0.5, window)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    cut, pieces = (2.0 ** -17.9, 3) if dtype == BF else (2.0 ** -21.9, 5)
    weights = np.where(many, 2.0 ** -7.9, 2.0 ** -13.9)[:, None, None] if dtype == BF else cut
    sums = 2.0 ** -24 * max(kv) / 64
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    bound = half * np.abs(out) + (2 * cut * b + 2.0 ** -18 * a + (pieces + 1) * sums)[..., None] * w + weights * W + 1e-30
    assert (np.abs(o - out) <= bound).all(), (np.abs(o - out) / bound).max()
    off = np.abs(lse - rl)
    assert (off <= cut * b + 2.0 ** -19 * a + 2.0 ** -17 + sums).all(), off.max()
    assert np.linalg.norm(o - out) <= (4e-3 if dtype == BF else 4e-6) * np.linalg.norm(out)
