"""Attention over the 8-bit cache where sequences of very different sizes share a
call, against the float64 reference (oracle/attention_oracle.py): what a row gets
does not depend on the rest of the batch or on how tight the caller's bounds are."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from tests.conftest import gpu_available
from tests.test_gpu_cache_attention import BF, F32, Setup, Twin, compare, queries

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


# ---------------------------------------------------------------------------
# bounds that are left out, too small, or passed by the offsets
# ---------------------------------------------------------------------------

def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("new", [[5, 1, 3], [40, 200, 1]])
def test_max_new_left_out(new):
    """With cu and no max_new any count of new tokens is taken."""
    import activation_sparse_ffn_amd as sffn
    s = Setup([90, 700, 33], 2, 64, 16, 31)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    q = queries(sum(new), 4, 64, BF, 32)
    batch = sffn.CacheBatch(i32(s.table), i32(s.kv), 700, cu)
    cache = s.cache()
    out, lse = sffn.cache_attention(cache, batch, q, out=torch.full_like(q, 7.0), return_lse=True)
    torch.cuda.synchronize()
    some_rows(s, out, lse, q, new, range(3))
    told = s.batch(new)
    x = torch.randn(sum(new), 2, 64, dtype=BF, device="cuda")
    sffn.kv_cache_append(cache, batch, x, x)
    for a, b in zip(sffn.kv_cache_read(cache, batch, sum(new)), sffn.kv_cache_read(cache, told, sum(new))):
        assert torch.equal(a, b) and (a.float() - x.float()).abs().max() < 0.05


def test_max_new_without_cu_is_one():
    import activation_sparse_ffn_amd as sffn
    s = Setup([9, 70], 2, 64, 16, 33)
    assert sffn.CacheBatch(i32(s.table), i32(s.kv), 70).max_new == 1


@pytest.mark.parametrize("H,most,max_kv", [
    (4, 1, 700), (4, 1, 90000),             # few rows, whole and in shares
    (8, 7, 700), (8, 7, 90000),             # two tiles of 16 rows
    (64, 3, 700), (64, 3, 90000),           # row tiles
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_beyond_max_new_are_nan(H, most, max_kv, dtype):
    import activation_sparse_ffn_amd as sffn
    new = [most, most + 9, 0, 2 * most]
    s = Setup([1900, 700, 33, 40], 2, 64, 16, 34)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    T = sum(new) + 2                        # the last two tokens are in no sequence
    q = queries(T, H, 64, dtype, 35)
    batch = sffn.CacheBatch(i32(s.table), i32(s.kv), max_kv, cu, most)
    out, lse = sffn.cache_attention(s.cache(), batch, q, out=torch.full_like(q, 7.0), return_lse=True)
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(new):
        m = min(n, most)
        if m:
            k, v = s.tokens(b)
            ref = ao.attend(q[at:at + m].double().cpu().numpy(), k, v, s.kv[b] - n, 0.125)
            compare(out[at:at + m], lse[at:at + m], ref, dtype)
        assert out[at + m:at + n].isnan().all() and lse[at + m:at + n].isnan().all()
        at += n
    assert (out[at:] == 7).all()


def test_tokens_beyond_max_new_above_the_shared_rows():
    import activation_sparse_ffn_amd as sffn
    new = [400, 300, 1]
    s = Setup([900, 310, 33], 2, 64, 64, 36)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    q = queries(701, 64, 64, BF, 37)
    out, lse = sffn.cache_attention(s.cache(), sffn.CacheBatch(i32(s.table), i32(s.kv), 900, cu, 290), q,
                                    out=torch.full_like(q, 7.0), return_lse=True)
    torch.cuda.synchronize()
    good = sffn.cache_attention(s.cache(), s.batch(new), q)
    bad = torch.zeros(701, dtype=torch.bool, device="cuda")
    bad[290:400] = bad[690:700] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert not out[~bad].isnan().any() and (out[~bad].float() - good[~bad].float()).abs().max() < 0.05


def test_sequences_that_run_out_of_the_call_are_nan():
    """cu beyond the call's tokens: the sequence's rows show it, in attention and in a
    read, and nothing is stored."""
    import activation_sparse_ffn_amd as sffn
    s = Setup([90, 70], 2, 64, 16, 38)
    for H in (4, 64):
        q = queries(7, H, 64, BF, 39)
        batch = sffn.CacheBatch(i32(s.table), i32(s.kv), 90, i32([0, 3, 9]), 6)
        out, lse = sffn.cache_attention(s.cache(), batch, q, out=torch.full_like(q, 7.0), return_lse=True)
        assert not out[:3].isnan().any() and out[3:].isnan().all() and lse[3:].isnan().all()
    cache = s.cache()
    before = [getattr(cache, n)[torch.from_numpy(s.table[1, :5])].clone() for n in ("keys", "values")]
    x = torch.randn(7, 2, 64, dtype=BF, device="cuda")
    sffn.kv_cache_append(cache, batch, x, x)
    for a, n in zip(before, ("keys", "values")):
        assert torch.equal(a, getattr(cache, n)[torch.from_numpy(s.table[1, :5])])
    k = torch.full((7, 2, 64), 7.0, dtype=BF, device="cuda")
    _, v = sffn.kv_cache_read(cache, batch, 7, k=k)
    assert not k[:3].isnan().any() and k[3:].isnan().all() and v[3:].isnan().all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("most", [1, 5, 17])
def test_append_and_read_take_max_new_tokens_and_no_more(page, most):
    import activation_sparse_ffn_amd as sffn
    kv, new = [100, 40], [30, 3]
    s = Setup(kv, 2, 64, page, 40)
    cu = i32([0, 30, 33])
    x = torch.randn(33, 2, 64, dtype=BF, device="cuda")
    few, all_ = s.cache(), s.cache()
    small = sffn.CacheBatch(i32(s.table), i32(kv), 100, cu, most)
    sffn.kv_cache_append(few, small, x, x)
    # the same first tokens as a call of their own
    m = [min(n, most) for n in new]
    part = sffn.CacheBatch(i32(s.table), i32([k - n + i for k, n, i in zip(kv, new, m)]), 100,
                           i32(np.concatenate([[0], np.cumsum(m)])), most)
    sffn.kv_cache_append(all_, part, torch.cat([x[:m[0]], x[30:30 + m[1]]]), torch.cat([x[:m[0]], x[30:30 + m[1]]]))
    for n in ("keys", "values", "k_scale", "v_scale"):
        a, b = getattr(few, n), getattr(all_, n)
        assert torch.equal(a.nan_to_num(-1) if a.is_floating_point() else a, b.nan_to_num(-1) if b.is_floating_point() else b), n
    out = torch.full((33, 2, 64), 7.0, dtype=BF, device="cuda")
    k, v = sffn.kv_cache_read(few, small, 33, k=out)
    full = sffn.kv_cache_read(few, s.batch(new), 33)
    for got, ref in zip((k, v), full):
        for a, n, i in ((0, 30, m[0]), (30, 3, m[1])):
            assert torch.equal(got[a:a + i], ref[a:a + i]) and got[a + i:a + n].isnan().all()


# ---------------------------------------------------------------------------
# append and read: a long prompt beside many sequences of a few tokens, whose pages
# have places by the call's tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,page,D", [(70, 16, 64), (300, 64, 128), (20, 32, 256)])
def test_append_of_a_prompt_beside_single_tokens(B, page, D, dtype):
    """Entries and scales bit for bit, some sequences with no new token."""
    rng = np.random.default_rng(B)
    held = rng.integers(0, 3 * page, B)
    t = Twin(held.tolist(), 2, D, page, seed=41, room=700)
    for step, (who, n) in enumerate(((B // 2, 650), (0, 600))):
        new = rng.integers(0, 4, B)
        new[who], new[B - 1] = n, 1
        t.append(new.tolist(), dtype, 42 + step, size=1.0 + step)
    s = t.s
    cu = np.concatenate([[0], np.cumsum(new)])
    batch = s.sffn.CacheBatch(i32(s.table), i32(t.kv), max(t.kv), i32(cu), int(new.max()))
    got = s.sffn.kv_cache_read(t.gpu, batch, int(cu[-1]), dtype)
    ref = [t.cpu.read(s.table[b], t.kv[b] - n, t.kv[b]) for b, n in enumerate(new)]
    for x, i in zip(got, (0, 1)):
        want = torch.from_numpy(np.concatenate([r[i] for r in ref]).astype(np.float32)).to(dtype)
        assert torch.equal(x.cpu(), want)


def test_append_beside_thousands_of_sequences():
    """5000 sequences (looked up in two steps): what calls of the single tokens and of
    the prompt alone store."""
    import activation_sparse_ffn_amd as sffn
    B, long_one, n, P = 5000, 3210, 900, 16
    rng = np.random.default_rng(43)
    kv = rng.integers(1, 40, B)
    kv[long_one] = n + 21
    s = Setup(kv.tolist(), 1, 64, P, 44)
    new = (rng.random(B) < 0.8).astype(int)
    new[long_one] = n
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    x = torch.randn(T, 1, 64, device="cuda")
    a, b = s.cache(), s.cache()
    sffn.kv_cache_append(a, sffn.CacheBatch(i32(s.table), i32(kv), 1000, i32(cu), n), x, x)
    at = int(cu[long_one])
    one = new.copy()
    one[long_one] = 0
    rest = torch.cat([x[:at], x[at + n:]])
    sffn.kv_cache_append(b, sffn.CacheBatch(i32(s.table), i32(kv), 1000, i32(np.concatenate([[0], np.cumsum(one)])), 1),
                         rest, rest)
    row = s.table[long_one:long_one + 1]
    sffn.kv_cache_append(b, sffn.CacheBatch(i32(row), i32([n + 21]), 1000, i32([0, n]), n), x[at:at + n], x[at:at + n])
    for name in ("keys", "values", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8)), name
    batch = sffn.CacheBatch(i32(s.table), i32(kv), 1000, i32(cu), n)
    k, v = sffn.kv_cache_read(a, batch, T, torch.float32)
    assert (k - x).abs().max() < 0.05 and (v - x).abs().max() < 0.05


def test_lost_tokens_among_many_sequences():
    """Beyond max_new, and behind the call's end, where pages have places by tokens."""
    import activation_sparse_ffn_amd as sffn
    B, P = 100, 16
    kv = [400] + [20] * (B - 1)
    s = Setup(kv, 1, 64, P, 45)
    new = [300] + [1] * (B - 1)
    cu = np.concatenate([[0], np.cumsum(new)])
    cu[-1] += 4                             # the last sequence leaves the call
    T = 300 + B - 1
    cache = s.cache()
    k = torch.full((T, 1, 64), 7.0, device="cuda")
    sffn.kv_cache_read(cache, sffn.CacheBatch(i32(s.table), i32(kv), 400, i32(cu), 290), T, torch.float32, k=k)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[290:300] = bad[-1] = True
    assert k[bad].isnan().all() and not k[~bad].isnan().any() and not (k[~bad] == 7).all()
    x = torch.full((T, 1, 64), 3.0, device="cuda")
    before = cache.keys[torch.from_numpy(s.table[B - 1, :2])].clone()
    sffn.kv_cache_append(cache, sffn.CacheBatch(i32(s.table), i32(kv), 400, i32(cu), 290), x, x)
    assert torch.equal(before, cache.keys[torch.from_numpy(s.table[B - 1, :2])])
    back, _ = sffn.kv_cache_read(cache, sffn.CacheBatch(i32(s.table), i32(kv), 400, i32(cu), 290), T, torch.float32)
    assert (back[~bad] - 3).abs().max() < 0.02


@pytest.mark.parametrize("much", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40])
def test_bounds_of_more_than_31_bits(much):
    """A window, max_new or max_kv past 31 bits means all, not its low bits."""
    import activation_sparse_ffn_amd as sffn
    s = Setup([300, 50], 2, 64, 16, 46)
    q = queries(6, 4, 64, BF, 47)
    cache, cu = s.cache(), i32([0, 4, 6])
    ref = sffn.cache_attention(cache, sffn.CacheBatch(i32(s.table), i32(s.kv), 300, cu, 6), q)
    got = sffn.cache_attention(cache, sffn.CacheBatch(i32(s.table), i32(s.kv), 300, cu, much), q,
                               out=torch.full_like(q, 7.0), window=much)
    assert torch.equal(got, ref)
    got = sffn.cache_attention(cache, sffn.CacheBatch(i32(s.table), i32(s.kv), much, cu, 6), q)
    assert (got.float() - ref.float()).abs().max() < 2.0 ** -6 * ref.float().abs().max()
    with pytest.raises(sffn.SparseFFNError):
        sffn.cache_attention(cache, sffn.CacheBatch(i32(s.table), i32(s.kv), 300, cu, 6), q, window=-much - 1)
    with pytest.raises(sffn.SparseFFNError):
        sffn.cache_attention(cache, sffn.CacheBatch(i32(s.table), i32(s.kv), 300, cu, -much - 1), q)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,n", [(4, 2), (8, 6), (8, 20), (8, 70)])
def test_lse_does_not_know_the_values(H, n, bad, dtype):
    """A page of values that are not finite shows in the rows that see it, not in the
    statistics, whichever kernel takes them (lse within 2^-17 + 2^-19 a of the reference,
    as everywhere: the scale's way through the exponent rounds differently)."""
    s = Setup([300], 2, 64, 16, 48)
    q = queries(n, H, 64, dtype, 49)
    good, _ = s.sffn.cache_attention(s.cache(), s.batch([n]), q, return_lse=True)
    k, v = s.tokens(0)
    _, ref, _, a = ao.attend(q.double().cpu().numpy(), k, v, 300 - n, 0.125)
    s.v_scale[s.table[0, 3], 0] = bad
    o, lse = s.sffn.cache_attention(s.cache(), s.batch([n]), q, return_lse=True)
    G = H // 2
    assert (np.abs(lse.double().cpu().numpy() - ref) <= 2.0 ** -17 + 2.0 ** -19 * a).all()
    assert torch.equal(o[:, G:], good[:, G:]) and not o[:, :G].isfinite().any()
