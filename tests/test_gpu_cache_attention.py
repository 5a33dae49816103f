"""The 8-bit cache and the attention over it on the GPU, against the float64
reference (oracle/attention_oracle.py).

The cache's arithmetic is defined in IEEE fp32, so its entries and scales are
compared bit for bit. Attention, with w = sum_j p_j |v_j| and a = max_j scale
sum_d |q_d k_jd| of the row, both from the reference: an fp32 score is off by at
most about 2^-21 a (rounding of sums of D <= 256 exact products; maximum and
exponent), so a weight by that much of itself; bf16 rounds each weight (2^-9)
and the result (2^-9), fp32 sums add under 2^-16 of w over these lengths:

  bf16  |o - ref| <= 2^-8 w + 2^-8 |ref| + 2^-19 a w       (twice the roundings)
  fp32  |o - ref| <= 2^-16 w + 2^-19 a w
  lse   |d| <= 2^-17 + 2^-19 a"""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Setup:
    """Sequences with kv[b] cached tokens in randomly chosen pages of a pool
    whose unused entries and scales are garbage (NaN scales)."""

    def __init__(self, kv, kv_heads, dim, page, seed=0, spare=3, loud=1.0):
        import activation_sparse_ffn_amd as sffn
        self.kv, self.K, self.D, self.P = list(kv), kv_heads, dim, page
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in kv]
        self.width = max(max(counts, default=0), 1) + 1
        total = sum(counts) + spare
        order = rng.permutation(total).tolist()
        self.table = np.full((len(kv), self.width), -7, np.int64)   # unused entries name no page
        for b, n in enumerate(counts):
            for i in range(n):
                self.table[b, i] = order.pop()
        self.keys = rng.integers(-127, 128, (total, kv_heads, page, dim)).astype(np.int8)
        self.values = rng.integers(-127, 128, (total, kv_heads, page, dim)).astype(np.int8)
        self.k_scale = (rng.uniform(0.2, 1.0, (total, kv_heads)) * loud / 73).astype(np.float32)
        self.v_scale = (rng.uniform(0.05, 1.0, (total, kv_heads)) / 73).astype(np.float32)
        self.k_scale[order], self.v_scale[order] = np.nan, np.nan
        self.spare = order
        self.sffn = sffn

    def cache(self):
        g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return self.sffn.KVCache(g(self.keys), g(self.values.transpose(0, 1, 3, 2)), g(self.k_scale), g(self.v_scale))

    def batch(self, new=None, max_kv=None, lens=None):
        lens = self.kv if lens is None else lens
        cu = None if new is None else i32(np.concatenate([[0], np.cumsum(new)]))
        return self.sffn.CacheBatch(i32(self.table), i32(lens), max(self.kv) if max_kv is None else max_kv, cu,
                                    1 if new is None else max(max(new, default=1), 1))

    def tokens(self, b):
        pos = np.arange(self.kv[b])
        pages, slots = self.table[b, pos // self.P], pos % self.P
        return (self.keys[pages, :, slots].astype(np.float64) * self.k_scale[pages][..., None],
                self.values[pages, :, slots].astype(np.float64) * self.v_scale[pages][..., None])


def queries(T, H, D, dtype, seed):
    return torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def compare(o, lse, ref, dtype):
    out, rl, w, a = ref
    o, lse, a3 = o.double().cpu().numpy(), lse.double().cpu().numpy(), a[..., None]
    bound = (2.0 ** -8 * (w + np.abs(out)) if dtype == BF else 2.0 ** -16 * w) + 2.0 ** -19 * a3 * w + 1e-30
    assert np.isfinite(o).all()
    worst = (np.abs(o - out) / bound).max() if out.size else 0
    assert worst <= 1, f"out: {worst:.2f} times the bound"
    none = np.isneginf(rl)
    assert (np.isneginf(lse) == none).all()
    assert (np.abs(lse - rl)[~none] <= (2.0 ** -17 + 2.0 ** -19 * a)[~none]).all()


def check(kv, new, H, K, D, page, dtype, window=0, scale=None, seed=0, max_kv=None, loud=1.0, q_view=False):
    s = Setup(kv, K, D, page, seed, loud=loud)
    n = [1] * len(kv) if new is None else new
    T = sum(n)
    q = queries(T, H + 3, D, dtype, seed + 1)
    q = q[:, 1:1 + H] if q_view else q[:, :H].contiguous()
    sc = D ** -0.5 if scale is None else scale
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new, max_kv), q, scale=scale, window=window, return_lse=True)
    torch.cuda.synchronize()
    refs, at = [], 0
    for b, m in enumerate(n):
        k, v = s.tokens(b)
        refs.append(ao.attend(q[at:at + m].double().cpu().numpy(), k, v, kv[b] - m, sc, window))
        at += m
    compare(o, lse, [np.concatenate(x) for x in zip(*refs)], dtype)


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
    ([70, 200], [33, 1], 4, 2, 64),                 # 4 waves
    ([97, 300, 3], [97, 64, 3], 6, 3, 32),
    ([333], [150], 4, 2, 128),                      # several row tiles
])
def test_several_tokens(kv, new, H, K, page, D, dtype):
    check(kv, new, H, K, D, page, dtype, seed=sum(new) + D)


@pytest.mark.parametrize("D", [64, 128])
def test_wide_row_tiles(D):
    """More than 128 rows of a sequence: the 8-wave workgroups, ragged."""
    check([290, 700, 129], [290, 91, 129], 7, 1, D, 64, BF, seed=5)
    check([600], [260], 2, 2, D, 16, BF, seed=6)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 100000])
def test_windows(window, dtype):
    check([333, 64, 1, 150], None, 4, 2, 64, 16, dtype, window=window, seed=window)
    check([333, 64, 150], [20, 64, 7], 6, 2, 64, 32, dtype, window=window, seed=window + 1)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_context_split_over_workgroups(dtype):
    check([9001], None, 4, 2, 128, 64, dtype, seed=1)
    check([9001, 17, 4000], None, 3, 1, 64, 16, dtype, seed=2)
    check([5003, 200], [40, 3], 4, 1, 64, 64, dtype, seed=3)
    check([5003], [9], 4, 4, 128, 32, dtype, window=1500, seed=4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 150])
def test_ragged_work_in_shares(window, D, dtype):
    """Drafts and chunks beside single tokens, cut across sequences, row tiles and
    heads: one tile of 16, two, one of 128, several."""
    check([2100, 33, 700], [5, 8, 3], 8, 2, D, 64, dtype, window=window, seed=1)
    check([1900, 40, 900], [20, 1, 3], 8, 2, D, 16, dtype, window=window, seed=2)
    check([1500, 40, 1200, 700], [300, 1, 64, 5], 6, 2, D, 32, dtype, window=window, seed=3)


@pytest.mark.parametrize("max_kv", [1, 300, 1500, 50000])
def test_shares_of_any_max_kv(max_kv):
    check([1500, 40, 1200, 700], [100, 1, 64, 5], 8, 2, 64, 32, BF, max_kv=max_kv, seed=4)
    check([1500] + [7 + i for i in range(70)], [6] + [3] * 70, 4, 1, 64, 16, BF, max_kv=max_kv, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (64, 100), (256, 0)])
def test_more_rows_than_are_shared(D, window, dtype):
    """Above 32768 rows: a workgroup for each tile and range of keys."""
    check([1100, 90], [490, 30], 64, 2, D, 64, dtype, window=window, seed=6)


def test_many_short_sequences():
    """Above 32768 rows, tiles of one sequence's few tokens, more than 64 sequences."""
    rng = np.random.default_rng(7)
    check(rng.integers(2, 90, 270).tolist(), [2] * 270, 64, 2, 64, 16, BF, seed=7)


@pytest.mark.parametrize("max_kv", [1, 64, 500, 100000])
def test_max_kv_never_changes_what_is_computed(max_kv):
    check([3000, 100], None, 4, 2, 64, 16, BF, seed=1, max_kv=max_kv)
    check([3000, 100], [20, 50], 4, 1, 64, 16, BF, seed=2, max_kv=max_kv)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores_and_other_scales(dtype):
    """Scores of some hundreds: the maximum has to be taken out."""
    check([200, 65], [1, 30], 4, 2, 64, 16, dtype, scale=1.0, loud=20.0, seed=1)
    check([200, 65], None, 4, 2, 64, 16, dtype, scale=-0.3, seed=2)
    check([200, 65], None, 4, 2, 64, 16, dtype, scale=0.0, seed=3)


def test_query_views():
    check([200, 65], [1, 30], 4, 2, 128, 64, BF, q_view=True, seed=1)
    check([200, 65], None, 4, 2, 128, 64, BF, q_view=True, seed=2)


# ---------------------------------------------------------------------------
# attention: rows, pages and values at the edges
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [2, 48])
def test_rows_that_see_nothing(H, dtype):
    """A sequence of no tokens, and one that holds fewer tokens than it has
    queries: those rows are zeros with lse -inf."""
    s = Setup([40, 5], 2, 64, 16, 1)
    q = queries(14, H, 64, dtype, 2)
    cache = s.cache()
    o, lse = s.sffn.cache_attention(cache, s.batch([1, 13], lens=[0, 5]), q, return_lse=True)
    torch.cuda.synchronize()
    assert (o[:9] == 0).all() and lse[:9].isneginf().all()
    k, v = s.tokens(1)
    ref = ao.attend(q[9:].double().cpu().numpy(), k, v, 0, 64 ** -0.5)
    compare(o[9:], lse[9:], ref, dtype)


def test_sequences_without_new_tokens_and_uncovered_rows():
    s = Setup([50, 60, 70], 1, 64, 16, 1)
    q = queries(7, 2, 64, BF, 2)
    cu = i32([0, 2, 2, 5])          # tokens 5 and 6 belong to no sequence
    batch = s.sffn.CacheBatch(i32(s.table), i32(s.kv), 70, cu, 3)
    for max_kv in (70, 9000):       # alone, and split over workgroups and joined
        batch = s.sffn.CacheBatch(i32(s.table), i32(s.kv), max_kv, cu, 3)
        out = torch.full_like(q, 7.0)
        s.sffn.cache_attention(s.cache(), batch, q, out=out)
        torch.cuda.synchronize()
        assert (out[5:] == 7).all()
        for b, a, e in ((0, 0, 2), (2, 2, 5)):
            k, v = s.tokens(b)
            ref = ao.attend(q[a:e].double().cpu().numpy(), k, v, s.kv[b] - (e - a), 0.125)
            compare(out[a:e], torch.from_numpy(ref[1]), ref, BF)


def test_no_tokens():
    s = Setup([50], 1, 64, 16, 1)
    q = queries(1, 2, 64, BF, 2)[:0]
    o, lse = s.sffn.cache_attention(s.cache(), s.batch([0]), q, return_lse=True)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)


@pytest.mark.parametrize("new", [None, [1, 40, 1]])
def test_pages_out_of_the_pool_show_in_their_rows_alone(new):
    """Entries that name no page, a table shorter than the sequence."""
    s = Setup([100, 90, 300], 1, 64, 16, 1)
    q = queries(3 if new is None else 42, 2, 64, BF, 2)
    good = s.sffn.cache_attention(s.cache(), s.batch(new), q)
    s.table[0, 2] = 1 << 30
    s.table[2, 18] = -1
    o = s.sffn.cache_attention(s.cache(), s.batch(new), q)
    mid = slice(1, 2 if new is None else 41)
    assert o[0].isnan().all() and o[-1].isnan().all() and torch.equal(o[mid], good[mid])
    o = s.sffn.cache_attention(s.cache(), s.batch(new, lens=[100, 90, 16 * s.width + 5]), q)
    assert o[-1].isnan().all() and torch.equal(o[mid], good[mid])
    # what lies behind a row's position or before its window does not matter
    s.table[2, 18] = -1
    o = s.sffn.cache_attention(s.cache(), s.batch(None, lens=[1, 90, 288]), q[:3].contiguous(), window=0)
    assert not o.isnan().any()
    o = s.sffn.cache_attention(s.cache(), s.batch(None, lens=[100, 90, 288]), q[:3].contiguous(), window=52)
    assert not o.isnan().any()


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_nan_scales_reach_only_rows_that_see_the_page(which):
    s = Setup([200], 2, 64, 16, 1)
    getattr(s, which)[s.table[0, 10], 1] = np.nan           # tokens 160 .. 175 of key head 1
    q = queries(60, 4, 64, BF, 2)                           # positions 140 .. 199
    o = s.sffn.cache_attention(s.cache(), s.batch([60]), q)
    assert not o[:, :2].isnan().any() and not o[:20].isnan().any() and o[20:, 2:].isnan().all()
    o = s.sffn.cache_attention(s.cache(), s.batch([60]), q, window=10)
    bad = torch.zeros(60, dtype=torch.bool)
    bad[20:45] = True                                       # 160 <= p < 175 + 10
    assert o[bad][:, 2:].isnan().all() and not o[~bad].isnan().any()


def test_queries_with_nan_and_infinity_stay_in_their_rows():
    s = Setup([200], 1, 64, 16, 1)
    q = queries(5, 2, 64, BF, 2)
    good = s.sffn.cache_attention(s.cache(), s.batch([5]), q)
    q[1, 0, 3], q[3, 1, 9] = float("nan"), float("inf")
    o = s.sffn.cache_attention(s.cache(), s.batch([5]), q)
    assert o[1, 0].isnan().all() and o[3, 1].isnan().all()
    same = torch.ones(5, 2, dtype=torch.bool)
    same[1, 0] = same[3, 1] = False
    assert torch.equal(o[same], good[same])


def test_zero_and_tiny_scales():
    s = Setup([100], 1, 64, 16, 1)
    s.v_scale[s.table[0, :3], 0] = [0.0, 1e-30, 1e30]
    s.k_scale[s.table[0, 4], 0] = 0.0
    q = queries(1, 2, 64, BF, 2)
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(), q, return_lse=True)
    k, v = s.tokens(0)
    compare(o, lse, ao.attend(q.double().cpu().numpy(), k, v, 99, 0.125), BF)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [2e-38, 1e-36, 1e-30, 1e-19, 1e28, 1e36])
@pytest.mark.parametrize("new,H", [([1, 3], 4), ([20, 33], 4), ([70, 90], 4)])
def test_value_scales_far_from_one(new, H, scale, dtype):
    """Every second page's values are scaled far down (or up): the statistics, which
    do not know the values, stay what they are, and so does every output that is
    finite in fp32 before it is divided."""
    s = Setup([300, 210], 2, 64, 16, 4)
    s.v_scale[::2] = scale
    q = queries(sum(new), H, 64, dtype, 5)
    o, lse = s.sffn.cache_attention(s.cache(), s.batch(new), q, return_lse=True)
    torch.cuda.synchronize()
    refs, at = [], 0
    for b, m in enumerate(new):
        k, v = s.tokens(b)
        refs.append(ao.attend(q[at:at + m].double().cpu().numpy(), k, v, s.kv[b] - m, 0.125))
        at += m
    ref = [np.concatenate(x) for x in zip(*refs)]
    if scale > 1e35:
        assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= 2.0 ** -17 + 2.0 ** -19 * ref[3]).all()
    else:
        compare(o, lse, ref, dtype)


def test_offsets_beyond_32_bits():
    """Pages behind 4 GiB of keys and of values."""
    import activation_sparse_ffn_amd as sffn
    pages, K, D, P = (1 << 32) // (8 * 64 * 128) + 40, 8, 128, 64
    cache = sffn.KVCache.empty(pages, K, D, P)
    small = Setup([150], K, D, P, 1, spare=0)
    ids = torch.tensor([pages - 1, pages - 20, pages - 7])
    for name, x in (("keys", small.keys), ("values", small.values.transpose(0, 1, 3, 2)),
                    ("k_scale", small.k_scale), ("v_scale", small.v_scale)):
        getattr(cache, name)[ids] = torch.from_numpy(np.ascontiguousarray(x[small.table[0, :3]])).cuda()
    table = i32(ids.tolist())[None]
    for n in (1, 50):
        q = queries(n, K, D, BF, 3)
        batch = sffn.CacheBatch(table, i32([150]), 150, i32([0, n]), n)
        o, lse = sffn.cache_attention(cache, batch, q, return_lse=True)
        k, v = small.tokens(0)
        compare(o, lse, ao.attend(q.double().cpu().numpy(), k, v, 150 - n, D ** -0.5), BF)
    x = torch.randn(2, K, D, dtype=BF, device="cuda")
    batch = sffn.CacheBatch(table, i32([152]), 152, i32([0, 2]), 2)
    sffn.kv_cache_append(cache, batch, x, x)
    k, v = sffn.kv_cache_read(cache, batch, 2)
    assert (k.float() - x.float()).abs().max() < 0.05 and (v.float() - x.float()).abs().max() < 0.05


# ---------------------------------------------------------------------------
# attention: repeats, streams, graphs
# ---------------------------------------------------------------------------

def test_same_bits_every_time_and_on_another_stream():
    s = Setup([3000, 100], 2, 64, 16, 1)
    cache, batch = s.cache(), s.batch([3, 40])
    q = queries(43, 4, 64, BF, 2)
    first = s.sffn.cache_attention(cache, batch, q)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(5):
            again = s.sffn.cache_attention(cache, batch, q)
    st.synchronize()
    assert torch.equal(first, again)


def test_graph_replays():
    """A decode step (rotation, append, attention) captured once and replayed
    with other inputs and lengths in the same buffers, against eager calls."""
    import activation_sparse_ffn_amd as sffn
    s = Setup([500, 41, 64], 2, 128, 16, 1)
    table = sffn.rope_table(1024, 128)
    bt, lens, pos = i32(s.table), i32([500, 41, 64]), i32([499, 40, 63])
    batch = sffn.CacheBatch(bt, lens, 600)
    q, k, v = queries(3, 8, 128, BF, 2), queries(3, 2, 128, BF, 3), queries(3, 2, 128, BF, 4)
    caches = [s.cache(), s.cache()]

    def step(cache):
        qq, kk = sffn.qk_norm_rope(q, k, pos, table, norm=True)
        sffn.kv_cache_append(cache, batch, kk, v)
        return sffn.cache_attention(cache, batch, qq)

    def fresh(i):
        lens.copy_(i32([500 + i, 41 + i, 64 - i]))
        pos.copy_(lens - 1)
        for t, seed in ((q, 5), (k, 6), (v, 7)):
            t.copy_(queries(*t.shape, BF, seed + 10 * i))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(s.cache())
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0])
    for n in ("keys", "values", "k_scale", "v_scale"):      # capture runs nothing; start alike all the same
        getattr(caches[0], n).copy_(getattr(caches[1], n))
    for i in range(4):
        fresh(i)
        graph.replay()
        eager = step(caches[1])
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        for n in ("keys", "values"):
            assert torch.equal(getattr(caches[0], n), getattr(caches[1], n))


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

class Twin:
    """The same sequences in the GPU's cache and the reference's."""

    def __init__(self, kv, K, D, page, seed=0, room=200):
        self.s = s = Setup([n + room for n in kv], K, D, page, seed)
        self.kv = list(kv)
        self.gpu, self.cpu = s.cache(), ao.Cache(len(s.keys), K, page, D)
        self.cpu.keys, self.cpu.values = s.keys.copy(), s.values.copy()
        self.cpu.k_scale, self.cpu.v_scale = s.k_scale.copy(), s.v_scale.copy()

    def append(self, new, dtype, seed, size=1.0, edit=None, cu=True):
        g = torch.Generator().manual_seed(seed)
        T, K, D = sum(new), self.s.K, self.s.D
        kv = torch.randn(T, 2 * K, D, generator=g) * size
        if edit is not None:
            edit(kv)
        kv = kv.to(dtype).cuda()
        k, v = kv[:, :K], kv[:, K:]
        self.kv = [a + b for a, b in zip(self.kv, new)]
        batch = self.s.sffn.CacheBatch(i32(self.s.table), i32(self.kv), max(self.kv),
                                       i32(np.concatenate([[0], np.cumsum(new)])) if cu else None, max(new))
        self.s.sffn.kv_cache_append(self.gpu, batch, k, v)
        at = 0
        for b, n in enumerate(new):
            self.cpu.append(self.s.table[b], self.kv[b] - n, k[at:at + n].float().cpu().numpy(),
                            v[at:at + n].float().cpu().numpy())
            at += n
        self.check()

    def check(self):
        """Scales of all pages, entries of every token stored, bit for bit."""
        torch.cuda.synchronize()
        for n in ("k_scale", "v_scale"):
            assert np.array_equal(getattr(self.gpu, n).cpu().numpy(), getattr(self.cpu, n), equal_nan=True), n
        keys, values = self.gpu.keys.cpu().numpy(), self.gpu.values.cpu().numpy().transpose(0, 1, 3, 2)
        for b, n in enumerate(self.kv):
            pos = np.arange(n)
            pages, slots = self.s.table[b, pos // self.s.P], pos % self.s.P
            assert np.array_equal(keys[pages, :, slots], self.cpu.keys[pages, :, slots])
            assert np.array_equal(values[pages, :, slots], self.cpu.values[pages, :, slots])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128), (128, 32), (64, 128)])
def test_append_bit_for_bit(D, page, dtype):
    t = Twin([0, 5, page, page - 1, 2 * page + 3], 2, D, page, seed=D)
    t.append([1, 1, 1, 1, 1], dtype, 1, cu=False)
    t.append([3, 0, 1, 40, 2], dtype, 2)
    t.append([100, 7, 0, 1, 16], dtype, 3, size=2.0)        # scales grow, held entries are rounded again
    t.append([1, 1, 1, 1, 1], dtype, 4, size=30.0, cu=False)
    t.append([5, 2, 9, 1, 33], dtype, 5, size=0.1)          # and stay where the new tokens are smaller


@pytest.mark.parametrize("page", [16, 64])
def test_append_of_zeros_tiny_and_non_finite_values(page):
    def zeros(x):
        x.zero_()

    def tiny(x):
        x.mul_(1e-44)

    def nan(x):
        x[1, 0, 3], x[2, 3, 5] = float("nan"), float("-inf")

    t = Twin([3, 0], 2, 64, page, seed=1)
    t.append([0, 4], F32, 1, edit=zeros)
    t.append([2, 2], F32, 2, edit=tiny)
    t.append([2, 3], BF, 3)
    t.append([3, 2], F32, 4, edit=nan)
    t.append([1, 2], F32, 5)
    t.append([page, page], F32, 6)          # the next pages are clean


def test_append_stores_nothing_outside_its_pages():
    t = Twin([20, 7], 1, 64, 16, seed=1, room=0)
    before = [getattr(t.gpu, n).clone() for n in ("keys", "values", "k_scale", "v_scale")]
    x = torch.randn(6, 1, 64, dtype=BF, device="cuda")
    s = t.s
    tab = s.table.copy()
    tab[0, 1], tab[1, 0] = 1 << 30, -3                      # no pages of the pool
    batch = s.sffn.CacheBatch(i32(tab), i32([23, 10]), 30, i32([0, 3, 6]), 3)
    s.sffn.kv_cache_append(t.gpu, batch, x, x)
    batch = s.sffn.CacheBatch(i32(s.table), i32([16 * s.width + 3, 0]), 30, i32([0, 3, 6]), 3)
    s.sffn.kv_cache_append(t.gpu, batch, x, x)              # behind the table's end; before position 0
    torch.cuda.synchronize()
    for a, n in zip(before, ("keys", "values", "k_scale", "v_scale")):
        assert torch.equal(a.view(torch.uint8), getattr(t.gpu, n).view(torch.uint8)), n
    k, v = s.sffn.kv_cache_read(t.gpu, batch, 6)
    assert k.isnan().all() and v.isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_read(D, page, dtype):
    s = Setup([1, page, 5 * page + 7, 2 * page - 1], 3, D, page, seed=2)
    new = [1, 3, 4 * page + 9, 0]
    got = s.sffn.kv_cache_read(s.cache(), s.batch(new), sum(new), dtype)
    for x, i in zip(got, (0, 1)):
        ref = np.concatenate([s.tokens(b)[i][s.kv[b] - n:] for b, n in enumerate(new)])
        want = torch.from_numpy(ref.astype(np.float32)).to(dtype)   # entry * scale, one fp32 product
        assert torch.equal(x.cpu(), want)
    heads = torch.empty(3, sum(new), D, dtype=dtype, device="cuda").transpose(0, 1)
    s.sffn.kv_cache_read(s.cache(), s.batch(new), sum(new), dtype, k=heads)
    assert torch.equal(heads, got[0])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals():
    s = Setup([50, 60], 2, 64, 16, 1)
    sffn, cache, batch = s.sffn, s.cache(), s.batch()
    q, x = queries(2, 4, 64, BF, 1), queries(2, 2, 64, BF, 2)
    tab, lens = i32(s.table), i32([50, 60])
    for bad in (lambda: sffn.cache_attention(cache, batch, q[..., :32]),
                lambda: sffn.cache_attention(cache, batch, q.half()),
                lambda: sffn.cache_attention(cache, batch, q.cpu()),
                lambda: sffn.cache_attention(cache, batch, q, out=q[:1]),
                lambda: sffn.cache_attention(cache, batch, q, workspace=torch.empty(8, device="cuda")),
                lambda: sffn.kv_cache_append(cache, batch, x, x.float()),
                lambda: sffn.kv_cache_append(cache, batch, x[:, :1], x[:, :1]),
                lambda: sffn.kv_cache_append(cache, batch, x, x[:1]),
                lambda: sffn.kv_cache_read(cache, batch, 2, torch.float16),
                lambda: sffn.KVCache(cache.keys, cache.keys, cache.k_scale, cache.v_scale),
                lambda: sffn.KVCache(cache.keys, cache.values, cache.k_scale[:1], cache.v_scale),
                lambda: sffn.KVCache(cache.keys.float(), cache.values, cache.k_scale, cache.v_scale),
                lambda: sffn.KVCache(cache.keys.cpu(), cache.values, cache.k_scale, cache.v_scale),
                lambda: sffn.CacheBatch(tab.long(), lens, 60),
                lambda: sffn.CacheBatch(tab, lens[:1], 60),
                lambda: sffn.CacheBatch(tab, lens, 60, i32([0, 2]))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sffn.cache_attention(cache, batch, q[:, :3]),          # 3 heads over 2
                lambda: sffn.cache_attention(cache, batch, q[:1]),             # 1 token, 2 sequences
                lambda: sffn.cache_attention(cache, batch, q, window=-1),
                lambda: sffn.cache_attention(cache, batch, q, scale=float("nan")),
                lambda: sffn.cache_attention(cache, batch, q, out=q[:1].expand(2, 4, 64)),
                lambda: sffn.cache_attention(cache, batch, queries(2, 4, 68, BF, 1)[..., 1:65]),
                lambda: sffn.kv_cache_append(cache, sffn.CacheBatch(tab, lens, 60, None, 0), x, x),
                lambda: sffn.kv_cache_append(sffn.KVCache.empty(4, 2, 96, 16), batch,
                                             queries(2, 2, 96, BF, 1), queries(2, 2, 96, BF, 2)),
                lambda: sffn.kv_cache_append(sffn.KVCache.empty(4, 2, 64, 24), batch, x, x)):
        with pytest.raises(sffn.SparseFFNError):
            bad()
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    long = sffn.CacheBatch(tab, lens, 30000)
    with pytest.raises(sffn.SparseFFNError, match="workspace"):
        sffn.cache_attention(cache, long, q, workspace=small)
