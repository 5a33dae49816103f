"""The 4-bit cache and attention over it on the GPU, against the float64 reference
(oracle/cache4_oracle.py).

Exponents, scales and entries are integer or IEEE fp32 arithmetic: equal bit for bit (signs
of zeros aside, which stand for the same). Attention, with w, W, a, b of the row as the
reference gives them: q is cut to 2^-17.9 (bf16, four pieces) or 2^-21.9 (fp32,
five) of the largest of its 32 channels, so a score is off by that times b and by fp32's
roundings, 2^-19 a; a weight and the sum each by that much of itself, twice that in their
quotient. Weights are cut to 2^-13.9 (three pieces; 2^-21.9 for fp32, five) of the largest of
32 that lie within 127 keys of each other, to 2^-7.9 in sequences of more than 128 rows: the
first of two pieces, whose largest lies in (3.75, 7.5] units and whose steps there are 1 / 2,
leaves up to 2^-2 units, the second's range ends at 7.5 / 32 = 2^-2 - 2^-6 units, and 2^-6 of
3.75 is 2^-7.9. The result is rounded by half a step; fp32 sums add 2^-16 of w over these
lengths.

  |o - ref| <= half |ref| + (2^-16.9 b + 2^-18 a + 2^-16) w + 2^-13.9 W    (bf16, few rows)
  |lse - ref| <= 2^-17.9 b + 2^-19 a + 2^-17"""
import numpy as np
import pytest
import torch

from oracle import cache4_oracle as co
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Setup:
    """Sequences with kv[b] cached tokens in randomly chosen pages of a pool whose unused
    rows are garbage (NaN scales, NaN exponents)."""

    def __init__(self, kv, kv_heads, dim, page, seed=0, spare=3, loud=0):
        import activation_sparse_ffn_amd as sffn
        self.sffn, self.kv, self.K, self.D, self.P = sffn, list(kv), kv_heads, dim, page
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in kv]
        self.width = max(max(counts, default=0), 1) + 1
        total = sum(counts) + spare
        order = rng.permutation(total).tolist()
        self.table = np.full((len(kv), self.width), -7, np.int64)       # unused entries name no page
        for b, n in enumerate(counts):
            for i in range(n):
                self.table[b, i] = order.pop()
        rows = (total, kv_heads, page)
        self.keys = rng.integers(0, 16, rows + (dim,)).astype(np.uint8)
        self.values = rng.integers(0, 16, rows + (dim,)).astype(np.uint8)
        self.k_exp = rng.integers(124 + loud, 127 + loud, rows + (dim // 32,)).astype(np.uint8)
        self.v_scale = rng.uniform(0.05, 0.5, rows).astype(np.float32)
        for b, n in enumerate(kv):
            if n % page:                            # behind the last token
                p = self.table[b, n // page]
                self.k_exp[p, :, n % page:], self.v_scale[p, :, n % page:] = 255, np.nan
        self.spare = order
        self.k_exp[order], self.v_scale[order] = 255, np.nan

    def cache(self):
        return self.sffn.KVCache4(gpu(co.pack(self.keys)), gpu(co.pack(self.values)), gpu(self.k_exp), gpu(self.v_scale))

    def batch(self, new=None, max_kv=None, lens=None, **kw):
        lens = self.kv if lens is None else lens
        cu = None if new is None else i32(np.concatenate([[0], np.cumsum(new)]))
        return self.sffn.CacheBatch(i32(self.table), i32(lens), max(self.kv) if max_kv is None else max_kv, cu,
                                    1 if new is None else max(max(new, default=1), 1), **kw)

    def tokens(self, b):
        """k, the codes and the scales of v of sequence b's tokens."""
        pos = np.arange(self.kv[b])
        p, s = self.table[b, pos // self.P], pos % self.P
        return co.key_values(self.keys[p, :, s], self.k_exp[p, :, s]), self.values[p, :, s], self.v_scale[p, :, s]


def queries(T, H, D, dtype, seed):
    return torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def reference(s, q, new, scale, window=0):
    """Of all tokens, and whether their sequence has more than 128 rows a key head."""
    refs, many, at = [], [], 0
    G = q.shape[1] // s.K
    for b, m in enumerate(new):
        if m:
            refs.append(co.attend(q[at:at + m].double().cpu().numpy(), *s.tokens(b), s.kv[b] - m, scale, window))
        many += [m * G > 128] * m
        at += m
    return [np.concatenate(x) for x in zip(*refs)], np.array(many)


def compare(o, lse, ref, many, dtype):
    out, rl, w, W, a, b = ref
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    cut = 2.0 ** -17.9 if dtype == BF else 2.0 ** -21.9
    weights = np.where(many, 2.0 ** -7.9, 2.0 ** -13.9)[:, None, None] if dtype == BF else cut
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    bound = half * np.abs(out) + (2 * cut * b + 2.0 ** -18 * a + 2.0 ** -16)[..., None] * w + weights * W + 1e-30
    assert np.isfinite(o).all()
    worst = (np.abs(o - out) / bound).max()
    assert worst <= 1, f"out: {worst:.2f} times the bound"
    none = np.isneginf(rl)
    assert (np.isneginf(lse) == none).all()
    assert (np.abs(lse - rl)[~none] <= (cut * b + 2.0 ** -19 * a + 2.0 ** -17)[~none]).all()
    # far from every rounding in one direction
    far = np.linalg.norm(o - out) / max(np.linalg.norm(out), 1e-30)
    assert far <= (4e-3 if dtype == BF else 4e-6), far


def check(kv, new, H, K, D, page, dtype, window=0, scale=None, seed=0, max_kv=None, q_view=False, loud=0):
    s = Setup(kv, K, D, page, seed, loud=loud)
    n = [1] * len(kv) if new is None else new
    T = sum(n)
    q = queries(T, H + 3, D, dtype, seed + 1)
    q = q[:, 1:1 + H] if q_view else q[:, :H].contiguous()
    sc = D ** -0.5 if scale is None else scale
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new, max_kv), q, scale=scale, window=window, return_lse=True)
    torch.cuda.synchronize()
    ref, many = reference(s, q, n, sc, window)
    compare(o, lse, ref, many, dtype)


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("by_slots", [False, True])
@pytest.mark.parametrize("kv,new,K,page", [([1], None, 1, 16), ([5, 64, 65, 130], None, 2, 64),
                                           ([40, 9, 130, 3], [3, 0, 70, 3], 3, 32), ([300], [299], 8, 128)])
def test_append_and_read(kv, new, K, page, D, dtype, by_slots):
    """Entries, exponents and scales of the new tokens; every other row as it was."""
    s = Setup(kv, K, D, page, 3)
    cache = s.cache()
    n = [1] * len(kv) if new is None else new
    T = sum(n)
    g = torch.Generator().manual_seed(T)
    loud = 1 + 30 * (torch.rand(D, generator=g) < 0.1)
    k, v = ((torch.randn(T, K + 1, D, generator=g) * loud * 10.0 ** torch.randint(-3, 4, (T, 1, 1), generator=g)).to(dtype).cuda()
            for _ in range(2))
    k, v = k[:, 1:], v[:, :K]
    batch = s.batch(new)
    if by_slots:
        batch = s.batch(new, slots=s.sffn.cache_slots(cache, batch, T)[1])
    s.sffn.kv_cache_append(cache, batch, k, v)
    kc, ke = co.quantise_keys(k.float().cpu().numpy())
    vc, vs = co.quantise_values(v.float().cpu().numpy())
    pos = np.concatenate([np.arange(m - c, m) for m, c in zip(kv, n)])
    seq = np.repeat(np.arange(len(kv)), n)
    p, i = s.table[seq, pos // page], pos % page
    s.keys[p, :, i], s.k_exp[p, :, i], s.values[p, :, i], s.v_scale[p, :, i] = kc, ke, vc, vs
    got = co.unpack(cache.keys.cpu().numpy()), co.unpack(cache.values.cpu().numpy())
    assert (co.decode(got[0]) == co.decode(s.keys)).all() and (co.decode(got[1]) == co.decode(s.values)).all()
    assert (cache.k_exp.cpu().numpy() == s.k_exp).all()
    np.testing.assert_array_equal(cache.v_scale.cpu().numpy(), s.v_scale)
    rk, rv = s.sffn.kv_cache_read(cache, batch, T, dtype)
    assert torch.equal(rk.cpu(), torch.from_numpy(co.key_values(kc, ke)).to(dtype))
    assert torch.equal(rv.cpu(), (torch.from_numpy(co.decode(vc)).float() * torch.from_numpy(vs)[..., None]).to(dtype))


def test_append_of_every_bf16_number():
    """Each in a block of its own with a neighbour a little larger and one smaller."""
    import activation_sparse_ffn_amd as sffn
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    k = torch.zeros(65536, 1, 64, dtype=torch.bfloat16)
    k[:, 0, 0], k[:, 0, 5], k[:, 0, 31] = x, x * 0.4, x * 0.07
    k[:, 0, 40] = x
    v = k.flip(2).contiguous()
    cache = sffn.KVCache4.empty(512, 1, 64, 128)
    slots = torch.randperm(65536, generator=torch.Generator().manual_seed(1)).cuda()
    batch = sffn.CacheBatch(i32(np.zeros((1, 1))), i32([1]), 1, slots=slots)
    sffn.kv_cache_append(cache, batch, k.cuda(), v.cuda())
    kc, ke = co.quantise_keys(k.float().numpy())
    vc, vs = co.quantise_values(v.float().numpy())
    at = slots.cpu().numpy()
    e = cache.k_exp.cpu().numpy().reshape(65536, 2)[at]
    assert (e == ke[:, 0]).all()
    fine = np.repeat(e != 255, 32, 1)
    got = co.unpack(cache.keys.cpu().numpy().reshape(65536, 32))[at]
    assert (co.decode(got) == co.decode(kc[:, 0]))[fine].all()
    sc = cache.v_scale.cpu().numpy().reshape(-1)[at]
    np.testing.assert_array_equal(sc, vs[:, 0])
    got = co.unpack(cache.values.cpu().numpy().reshape(65536, 32))[at]
    assert (co.decode(got) == co.decode(vc[:, 0]))[np.isfinite(sc)].all()


def test_tokens_without_a_slot():
    """Slots outside the pool, tokens beyond max_new, unknown pages: nothing is stored, a read
    shows NaN; rows of tokens in no sequence stay as they are."""
    s = Setup([20, 40], 2, 64, 16, 1)
    cache = s.cache()
    before = [t.clone() for t in (cache.keys, cache.values, cache.k_exp, cache.v_scale)]
    k = torch.randn(7, 2, 64, device="cuda")
    bad = torch.tensor([-1, -5, cache.keys.shape[0] * 16, 1 << 40, -(1 << 62), (1 << 63) - 1, -1], device="cuda")
    s.sffn.kv_cache_append(cache, s.batch([3, 4], slots=bad), k, k)
    lost = s.sffn.CacheBatch(i32(np.full((2, 3), 999)), i32([20, 40]), 40, i32([0, 3, 7]), 4)
    s.sffn.kv_cache_append(cache, lost, k, k)
    for a, b in zip(before, (cache.keys, cache.values, cache.k_exp, cache.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = torch.full((9, 2, 64), 5.0, device="cuda")
    rk, rv = s.sffn.kv_cache_read(cache, s.sffn.CacheBatch(i32(s.table), i32([20, 40]), 40, i32([1, 3, 7]), 3), 9, F32,
                                  k=out.clone(), v=out.clone())
    for r in (rk, rv):
        assert (r[0] == 5).all() and (r[7:] == 5).all() and r[6].isnan().all() and torch.isfinite(r[1:6]).all()
    rk, _ = s.sffn.kv_cache_read(cache, lost, 7, F32)
    assert rk.isnan().all()


# ---------------------------------------------------------------------------
# attention: values
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,H,K,page", [
    ([1], 1, 1, 16),
    ([1, 2, 15, 16, 17], 4, 2, 16),
    ([63, 64, 65, 127, 128, 129], 8, 2, 64),
    ([300, 5, 1, 777], 7, 1, 32),
    ([255, 400], 16, 1, 128),
    ([90, 33], 24, 1, 64),          # more than 16 rows for one token
])
def test_single_tokens(kv, H, K, page, D, dtype):
    check(kv, None, H, K, D, page, dtype, seed=len(kv) + D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv,new,H,K,page", [
    ([5], [5], 1, 1, 16),
    ([40, 9, 130], [3, 1, 2], 4, 1, 16),            # drafts: few rows
    ([70, 200], [33, 1], 4, 2, 64),
    ([97, 300, 3], [97, 64, 3], 6, 3, 32),
    ([333], [150], 4, 2, 128),                      # several row tiles
    ([200, 0, 65], [200, 0, 1], 3, 1, 64),          # nothing cached, an empty sequence
])
def test_chunks(kv, new, H, K, page, D, dtype):
    check(kv, new, H, K, D, page, dtype, seed=len(kv) + D, q_view=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 15, 64, 100, 1000])
@pytest.mark.parametrize("kv,new,H,K", [([700, 30, 129], None, 4, 2), ([400, 90], [7, 90], 8, 2), ([500], [300], 2, 1)])
def test_windows(kv, new, H, K, window, D, dtype):
    check(kv, new, H, K, D, 32, dtype, window=window, seed=window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [None, [150]])
@pytest.mark.parametrize("scale,loud", [(0.0, 0), (-0.2, 0), (1.0, 0), (0.05, 6), (3.0, 0)])
def test_scales(scale, loud, new, dtype):
    """Zero, negative and large ones: scores to hundreds, which leave one key all the weight."""
    check([500], new, 4, 2, 128, 64, dtype, scale=scale, seed=5, loud=loud)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv,H,K,D,max_kv", [([5000], 8, 2, 128, None), ([20000], 2, 2, 64, None), ([3000, 100, 9000], 4, 1, 128, 1),
                                             ([6000], 4, 1, 256, 1 << 30)])
def test_long_sequences_in_parts(kv, H, K, D, max_kv, dtype):
    check(kv, None, H, K, D, 64, dtype, seed=D, max_kv=max_kv)
    check(kv, [3] * len(kv), H, K, D, 64, dtype, seed=D + 1, max_kv=max_kv)


def test_many_rows_over_many_keys():
    check([3000, 2500], [40, 33], 8, 1, 128, 64, BF, seed=1)
    check([2000], [2], 64, 1, 128, 128, BF, seed=2)


# ---------------------------------------------------------------------------
# attention: what rows do not see, and see
# ---------------------------------------------------------------------------

def attend(s, q, new, **kw):
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new), q, return_lse=True, **kw)
    torch.cuda.synchronize()
    return o.float().cpu().numpy(), lse.cpu().numpy()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H", [4, 48])
def test_nan_is_seen_by_the_rows_that_see_it(H, D):
    """A NaN exponent or scale of one key makes the rows NaN that see it, and those alone."""
    new, kv = [40], [300]
    s = Setup(kv, 2, D, 16, 7)
    q = queries(40, H, D, BF, 1)
    clean, _ = attend(s, q, new)
    at = 280                                # seen by tokens 280 .. 299, the last 20
    p, i = s.table[0, at // 16], at % 16
    for name, where in (("k_exp", (p, 1, i, D // 32 - 1)), ("v_scale", (p, 1, i))):
        t = Setup(kv, 2, D, 16, 7)
        getattr(t, name)[where] = 255 if name == "k_exp" else np.nan
        o, lse = attend(t, q, new)
        assert np.isnan(o[20:, H // 2:]).all() and (o[:20] == clean[:20]).all() and (o[:, :H // 2] == clean[:, :H // 2]).all()
        if name == "k_exp":
            assert np.isnan(lse[20:, H // 2:]).all()
        else:
            assert np.isfinite(lse).all()
        assert np.isfinite(lse[:20]).all()
    # window: the rows behind it no longer see the key
    t = Setup(kv, 2, D, 16, 7)
    t.v_scale[p, :, i] = np.nan
    o, _ = attend(t, q, new, window=10)
    assert np.isnan(o[20:30]).all() and np.isfinite(o[:20]).all() and np.isfinite(o[30:]).all()


@pytest.mark.parametrize("new", [[1], [90]])
def test_queries_that_are_not_finite(new):
    s = Setup([200], 1, 128, 64, 3)
    q = queries(new[0], 4, 128, BF, 1)
    clean, _ = attend(s, q, new)
    q[0, 1, 77], q[0, 2, 0] = float("nan"), float("inf")
    o, _ = attend(s, q, new)
    assert np.isnan(o[0, 1]).all() and np.isnan(o[0, 2]).all()
    o[0, 1:3] = clean[0, 1:3]
    assert (o == clean).all()


@pytest.mark.parametrize("new", [[1], [90]])
def test_pages_that_are_unknown(new):
    for bad in (-1, 999, 2 ** 31 - 1, -2 ** 31):
        s = Setup([200, 100], 2, 64, 32, 3)
        s.table[0, 2] = bad
        o, lse = attend(s, queries(2 * new[0], 4, 64, BF, 1), [new[0]] * 2)
        assert np.isfinite(o[new[0]:]).all()
        seen = np.arange(200 - new[0], 200) >= 64
        assert np.isnan(o[:new[0]][seen]).all() and np.isfinite(o[:new[0]][~seen]).all()
    # more tokens than the table has room for
    s = Setup([64], 1, 64, 32, 3)
    o = s.sffn.cache_attention(s.cache(), s.batch(lens=[200]), queries(1, 4, 64, BF, 1))
    assert o.isnan().all()


def test_values_of_very_unlike_scales():
    """A hidden key of a huge scale, and a seen one of a tiny, take nothing from the others."""
    for new in ([1], [140]):
        s = Setup([300], 1, 128, 64, 11)
        base, many = reference(s, q := queries(new[0], 4, 128, BF, 2), new, 128 ** -0.5)
        pos = np.arange(300)
        s.v_scale[s.table[0, pos[::7] // 64], :, pos[::7] % 64] *= 1e-30
        s.v_scale[s.table[0, 4], :, 300 % 64:] = 1e38
        ref, many = reference(s, q, new, 128 ** -0.5)
        o, lse = s.sffn.cache_attention(s.cache(), s.batch(new), q, return_lse=True)
        compare(o, lse, ref, many, BF)


def test_rows_that_see_nothing_and_rows_of_no_sequence():
    s = Setup([5, 0, 9], 2, 64, 16, 1)
    q = queries(6, 4, 64, BF, 1)
    out = torch.full((6, 4, 64), 3.0, dtype=BF, device="cuda")
    # sequence 1 says it holds nothing, yet two tokens of the call are its: they see no key
    batch = s.sffn.CacheBatch(i32(s.table), i32([5, 0, 9]), 9, i32([0, 1, 3, 4]), 2)
    o, lse = s.sffn.cache_attention(s.cache(), batch, q, out=out, return_lse=True)
    assert o is out and (o[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()
    assert (o[4:] == 3).all() and torch.isfinite(o[[0, 3]].float()).all()
    # beyond max_new: NaN
    batch = s.sffn.CacheBatch(i32(s.table), i32([5, 0, 9]), 9, i32([0, 1, 1, 6]), 3)
    o = s.sffn.cache_attention(s.cache(), batch, q, out=torch.full_like(out, 3.0))
    assert o[4:].isnan().all() and torch.isfinite(o[1:4].float()).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("new", [1, 5, 64])
def test_repeated_captured_and_on_another_stream(new):
    s = Setup([900, 40, 3000], 2, 128, 64, 5)
    cache, n = s.cache(), [new, min(new, 40), new]
    batch = s.batch(n)
    T = sum(n)
    q = queries(T, 8, 128, BF, 3)
    k, v = queries(T, 2, 128, BF, 4), queries(T, 2, 128, BF, 5)

    def call():
        s.sffn.kv_cache_append(cache, batch, k, v)
        o, lse = s.sffn.cache_attention(cache, batch, q, return_lse=True)
        return [*s.sffn.kv_cache_read(cache, batch, T), o, lse]

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
        s.sffn.cache_attention(cache, batch, q)


def test_a_workspace_of_the_callers():
    s = Setup([4000], 2, 128, 64, 5)
    q = queries(1, 8, 128, BF, 3)
    cache, batch = s.cache(), s.batch()
    want = s.sffn.cache_attention(cache, batch, q)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(s.sffn.cache_attention(cache, batch, q, workspace=ws), want)
    with pytest.raises(s.sffn.SparseFFNError):
        s.sffn.cache_attention(cache, batch, q, workspace=ws[:256])


def test_both_caches_in_a_step_of_a_planned_batch():
    """Plan, append by slots, attention: as a model runs them, over steps; the 4-bit cache's
    attention is the reference's over what it holds."""
    import activation_sparse_ffn_amd as sffn
    page, K, D, H = 16, 2, 64, 4
    free, n_free = sffn.free_pages(40)
    table = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    lens = i32([0, 0, 0])
    caches = sffn.KVCache4.empty(40, K, D, page), sffn.KVCache.empty(40, K, D, page)
    ks, vs = [[], [], []], [[], [], []]
    for step, new in enumerate([[20, 5, 33], [1, 1, 1], [17, 0, 2], [1, 1, 1]]):
        T = sum(new)
        plan = sffn.page_plan(table, lens, i32(new), free, n_free, page, T)
        lens, n_free = plan.kv_lens, plan.n_free
        batch = sffn.CacheBatch(table, lens, 200, plan.cu, max(new), slots=plan.slots)
        k, v, q = (queries(T, h, D, F32, 10 * step + i) for i, h in enumerate((K, K, H)))
        outs = []
        for cache in caches:
            sffn.kv_cache_append(cache, batch, k, v)
            outs.append(sffn.cache_attention(cache, batch, q, return_lse=True))
        at = 0
        for b, m in enumerate(new):
            ks[b].append(k[at:at + m].cpu().numpy())
            vs[b].append(v[at:at + m].cpu().numpy())
            if m:
                kc, ke = co.quantise_keys(np.concatenate(ks[b]))
                vc, sc = co.quantise_values(np.concatenate(vs[b]))
                ref = co.attend(q[at:at + m].double().cpu().numpy(), co.key_values(kc, ke), vc, sc, kc.shape[0] - m, D ** -0.5)
                compare(outs[0][0][at:at + m], outs[0][1][at:at + m], ref, np.array([False] * m), F32)
            at += m
    # 4 bits keep about a tenth of each entry, 8 about a hundredth
    assert (outs[0][0] - outs[1][0]).norm() < 0.3 * outs[1][0].norm()


def test_pages_beyond_4_gib():
    """The last pages of a pool of more than 2^32 bytes of keys and of values: append, read and
    attention as over the first pages of a small one."""
    import activation_sparse_ffn_amd as sffn
    K, D, P, big = 8, 256, 128, 34000
    g = torch.Generator(device="cuda").manual_seed(4)
    new, T = [300, 1], 301
    k, v = (torch.randn(T, K, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, 2 * K, D, generator=g, device="cuda").bfloat16()
    outs = []
    for pages in (8, big):
        cache = sffn.KVCache4.empty(pages, K, D, P)
        assert pages == 8 or cache.keys.numel() > 1 << 32
        table = i32([[pages - 1, pages - 2, pages - 3], [pages - 4, 0, 0]])
        batch = sffn.CacheBatch(table, i32([300, 1]), 300, i32([0, 300, 301]), 300)
        _, slots = sffn.cache_slots(cache, batch, T)
        assert slots[0] == (pages - 1) * P
        sffn.kv_cache_append(cache, sffn.CacheBatch(table, i32([300, 1]), 300, i32([0, 300, 301]), 300, slots=slots), k, v)
        chunk = sffn.cache_attention(cache, batch, q)
        one = sffn.cache_attention(cache, sffn.CacheBatch(table, i32([300, 1]), 300), q[[299, 300]])
        outs.append((*sffn.kv_cache_read(cache, batch, T), chunk, one))
        del cache
    for a, b in zip(*outs):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("max_kv", [1, 500, 3000, 60000])
def test_one_sequence_cut_by_any_length(max_kv, window):
    """max_kv cuts one sequence's row tiles into ranges of keys; what is computed is the same."""
    check([3000], [70], 8, 2, 128, 64, BF, window=window, seed=21, max_kv=max_kv)
    check([1300], [41], 4, 1, 64, 16, F32, window=window, seed=22, max_kv=max_kv)
