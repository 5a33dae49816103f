"""Attention over the 8-bit cache where sequences of very different sizes share a
call, against the float64 reference (oracle/attention_oracle.py): what a row gets
does not depend on the rest of the batch or on how tight the caller's bounds are."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from tests.conftest import gpu_available
from tests.test_gpu_cache_attention import BF, F32, Setup, compare, queries

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def close_to_16_bit_weights(o, q, s, b, p0, scale):
    """Rows of sequence b, whose weights are two bf16 pieces. A piece holds 8 bits, so
    a weight is off by 2^-16 of itself at most; fp32 scores and sums add less than
    2^-19 a and 2^-16. With w = sum_j p_j |v_j| and a the largest sum of a score's
    terms, a value within r = (2^-15 + 2^-19 a) w of the exact one is rounded to bf16:

      bf16(ref - r) <= o <= bf16(ref + r)

    One piece (up to 2^-8 of each weight) leaves that wherever |ref| is well below w."""
    k, v = s.tokens(b)
    ref, _, w, a = ao.attend(q.double().cpu().numpy(), k, v, p0, scale)
    r = (2.0 ** -15 + 2.0 ** -19 * a[..., None]) * w
    lo, hi = (torch.from_numpy(x).bfloat16().double().numpy() for x in (ref - r, ref + r))
    o = o.double().cpu().numpy()
    out = (o < lo) | (o > hi)
    assert not out.any(), f"sequence {b}: {out.sum()} of {out.size} outside"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,chunk", [(8, 150), (32, 600)])      # in shares; above 32768 rows for H 64 below
def test_single_tokens_beside_a_chunk_are_as_exact_as_alone(H, chunk, D):
    """Sequences of 1, 3 and 32 tokens (128 rows of 4 heads) beside a chunk."""
    new = [1, chunk, 3, 1, 128 // (H // 2)]
    s = Setup([700, chunk + 40, 90, 7, 333], 2, D, 64, 11)
    q = queries(sum(new), H, D, BF, 12)
    o = s.sffn.cache_attention(s.cache(), s.batch(new), q)
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(new):
        if b != 1:
            close_to_16_bit_weights(o[at:at + n], q[at:at + n], s, b, s.kv[b] - n, D ** -0.5)
        at += n


@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens_beside_a_chunk_of_more_rows_than_are_shared(D):
    new = [1, 600, 2]
    s = Setup([700, 640, 90], 2, D, 64, 13)
    q = queries(sum(new), 64, D, BF, 14)
    assert q.shape[0] * 64 > 32768
    o = s.sffn.cache_attention(s.cache(), s.batch(new), q)
    torch.cuda.synchronize()
    close_to_16_bit_weights(o[:1], q[:1], s, 0, 699, D ** -0.5)
    close_to_16_bit_weights(o[601:], q[601:], s, 2, 88, D ** -0.5)


@pytest.mark.parametrize("max_new", [1, 9, 40, 5000])
def test_a_generous_max_new_costs_no_precision(max_new):
    import activation_sparse_ffn_amd as sffn
    s = Setup([700, 90], 2, 128, 64, 15)
    q = queries(2, 8, 128, BF, 16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    batch = sffn.CacheBatch(i32(s.table), i32(s.kv), 700, i32([0, 1, 2]), max_new)
    o = sffn.cache_attention(s.cache(), batch, q)
    torch.cuda.synchronize()
    for b in range(2):
        close_to_16_bit_weights(o[b:b + 1], q[b:b + 1], s, b, s.kv[b] - 1, 128 ** -0.5)


@pytest.mark.parametrize("H", [8, 64])
def test_the_same_bits_every_time_for_chunks_and_single_tokens(H):
    new = [1, 600, 3]
    s = Setup([2700, 900, 90], 2, 128, 64, 17)
    q = queries(sum(new), H, 128, BF, 18)
    cache, batch = s.cache(), s.batch(new)
    first = s.sffn.cache_attention(cache, batch, q, return_lse=True)
    for _ in range(4):
        again = s.sffn.cache_attention(cache, batch, q, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ---------------------------------------------------------------------------
# many sequences: rows have fewer parts than their keys would fill, or one
# ---------------------------------------------------------------------------

def some_rows(s, o, lse, q, new, which):
    """Sequences `which` against the reference (the bounds of test_gpu_cache_attention)."""
    at = np.concatenate([[0], np.cumsum(new)])
    for b in which:
        a, e = at[b], at[b + 1]
        k, v = s.tokens(b)
        ref = ao.attend(q[a:e].double().cpu().numpy(), k, v, s.kv[b] - new[b], s.D ** -0.5)
        compare(o[a:e], lse[a:e], ref, q.dtype)


@pytest.mark.parametrize("B,H,dtype,parts", [(1000, 16, BF, 16), (4200, 32, BF, 1), (4200, 32, F32, 1)])
def test_one_long_sequence_among_many_short_ones(B, H, dtype, parts):
    """1000 sequences of 16 rows of 256 channels leave room for 16 parts a row: the
    longest sequence is cut into fewer than its 40 shares; 4200 of 32 heads leave none."""
    rng = np.random.default_rng(21)
    kv = rng.integers(1, 60, B)
    kv[B // 3] = 20000
    s = Setup(kv.tolist(), H // 16, 256, 128, 22)
    q = queries(B, H, 256, dtype, 23)
    cache, batch = s.cache(), s.batch(max_kv=20000)
    lib = s.sffn.load_library()
    need = lib.cache_attention_workspace_size(cache._c, batch._c, H, int(dtype is BF), 0, B)
    assert need == (0 if parts == 1 else B * H * (parts * 258 + 1) * 4)
    o, lse = s.sffn.cache_attention(cache, batch, q, return_lse=True)
    torch.cuda.synchronize()
    some_rows(s, o, lse, q, [1] * B, [0, 1, B // 3 - 1, B // 3, B // 3 + 1, B // 2, B - 2, B - 1])


def test_drafts_of_many_sequences():
    """Two tiles of 16 rows (8 tokens of 4 heads) in 400 sequences, 25600 rows."""
    rng = np.random.default_rng(24)
    kv = rng.integers(8, 100, 400)
    kv[[5, 399]] = [9000, 4000]
    s = Setup(kv.tolist(), 2, 128, 64, 25)
    new = [8] * 400
    q = queries(3200, 8, 128, BF, 26)
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new), q, return_lse=True)
    torch.cuda.synchronize()
    some_rows(s, o, lse, q, new, [0, 4, 5, 6, 200, 398, 399])
