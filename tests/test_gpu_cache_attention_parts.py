"""Attention over the 8-bit cache where a row's keys are cut into several parts that
are joined: the edges of rows, pages, scales and values, in every kernel. The
reference is float64 on the GPU, checked against the one of oracle/attention_oracle.py;
bounds are those of tests/test_gpu_cache_attention.py."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as ao
from tests.conftest import gpu_available
from tests.test_gpu_cache_attention import BF, F32, Setup, compare, queries

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

# (query heads, new tokens, cached tokens) of sequences with 2 key heads: the rows of a
# sequence and key head choose the kernel. (Above 32768 rows a row has several parts
# only where tiles are of 256 rows: bf16, heads of up to 128.)
CASES = {
    "few": (4, [1, 3, 1], [3000, 1700, 9]),             # a tile of 16 rows
    "pair": (8, [6, 2, 8], [3000, 1700, 9]),            # two of them
    "rows": (8, [20, 5, 1], [3000, 1700, 9]),           # row tiles of 128
    "many": (8, [60, 1, 7], [3000, 1700, 9]),           # of 256 (fp32: of 128)
    "unshared": (64, [520], [3000]),                    # above 32768 rows: ranges of keys
}
every_kernel = pytest.mark.parametrize("case", list(CASES))
both = pytest.mark.parametrize("dtype", [BF, F32])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend64(q, k, v, p0, scale, window=0):
    """As ao.attend, on the GPU."""
    n, H, D = q.shape
    L, K, _ = k.shape
    q, k, v = q.double(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    p, j = torch.arange(p0, p0 + n, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
    sees = (j <= p) & (j > p - window if window else j >= 0)
    none = ~sees.any(1)
    out, weight = torch.zeros_like(q), torch.zeros_like(q)
    lse, size = torch.full((n, H), -np.inf, dtype=q.dtype, device="cuda"), torch.zeros(n, H, dtype=q.dtype, device="cuda")
    for h in range(H):
        kh, vh = k[:, h * K // H], v[:, h * K // H]
        s = (scale * (q[:, h].contiguous() @ kh.t().contiguous())).masked_fill(~sees, -np.inf)
        w = torch.softmax(s, 1).masked_fill(none[:, None], 0)
        out[:, h], weight[:, h] = w @ vh.contiguous(), w @ vh.abs().contiguous()
        lse[:, h] = torch.logsumexp(s, 1)
        terms = abs(scale) * (q[:, h].abs().contiguous() @ kh.abs().t().contiguous())
        size[:, h] = terms.masked_fill(~sees, 0).amax(1)
    return [x.cpu().numpy() for x in (out, lse, weight, size)]


def test_the_reference_is_the_oracle():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    for p0, window in ((4, 0), (4, 3), (-2, 0)):
        got = attend64(torch.from_numpy(q).cuda(), k, v, p0, 0.3, window)
        for a, b in zip(got, ao.attend(q, k, v, p0, 0.3, window)):
            assert np.allclose(a, b, atol=1e-12)


class Call:
    """One of CASES with D channels, its pages and queries; run() returns out and lse
    and asserts that the rows of the long sequences have several parts."""

    def __init__(self, case, dtype, D=64, page=16, seed=1):
        self.case = case
        self.H, self.new, self.kv = CASES[case]
        self.s = Setup(self.kv, 2, D, page, seed)
        self.dtype, self.scale = dtype, D ** -0.5
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.q = queries(self.cu[-1], self.H, D, dtype, seed + 1)

    def run(self, window=0, lens=None, cu=None, q=None, out=None, several=True):
        s, q = self.s, self.q if q is None else q
        cache = s.cache()
        batch = s.sffn.CacheBatch(i32(s.table), i32(self.kv if lens is None else lens), max(self.kv),
                                  i32(self.cu if cu is None else cu), max(self.new))
        need = s.sffn.load_library().cache_attention_workspace_size(cache._c, batch._c, self.H, int(self.dtype is BF),
                                                                    window, q.shape[0])
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")     # NaN, and -1 for the counts of parts
        o, lse = s.sffn.cache_attention(cache, batch, q, window=window, out=out, return_lse=True,
                                        workspace=ws if need else None)
        torch.cuda.synchronize()
        if several and not (self.case == "unshared" and (self.dtype is F32 or s.D == 256)):
            parts = ws.view(torch.int32)[-q.shape[0] * self.H:].view(q.shape[0], self.H)
            assert (parts[:self.new[0]] > 1).all()
        return o, lse

    def rows(self, b):
        return slice(int(self.cu[b]), int(self.cu[b + 1]))

    def check(self, o, lse, which, window=0):
        for b in which:
            k, v = self.s.tokens(b)
            r = self.rows(b)
            ref = attend64(self.q[r], k, v, self.kv[b] - self.new[b], self.scale, window)
            compare(o[r], lse[r], ref, self.dtype)


@both
@every_kernel
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 128)])
def test_values(case, D, page, dtype):
    c = Call(case, dtype, D, page)
    c.check(*c.run(), range(len(c.kv)))
    c.check(*c.run(window=1200), range(len(c.kv)), 1200)


@both
@pytest.mark.parametrize("H,n", [(4, 1200), (64, 1200)])
def test_rows_that_see_nothing_in_a_tile_that_sees_much(H, n, dtype):
    """1200 queries of a sequence that holds 1000 tokens: the first 200 see none, the
    others of their row tiles see up to 1000."""
    s = Setup([1000, 3], 2, 64, 16, 2)
    q = queries(n + 2, H, 64, dtype, 3)
    batch = s.sffn.CacheBatch(i32(s.table), i32([1000, 0]), 1000, i32([0, n, n + 2]), n)
    o, lse = s.sffn.cache_attention(s.cache(), batch, q, return_lse=True)
    torch.cuda.synchronize()
    for r in (slice(0, 200), slice(n, n + 2)):
        assert (o[r] == 0).all() and lse[r].isneginf().all()
    k, v = s.tokens(0)
    compare(o[:n], lse[:n], attend64(q[:n], k, v, -200, 0.125), dtype)


@both
@every_kernel
def test_tokens_of_no_sequence_and_sequences_of_no_token(case, dtype):
    c = Call(case, dtype)
    new, T = [n if b != 1 else 0 for b, n in enumerate(c.new)], int(c.cu[-1])
    q = torch.cat([c.q, c.q[:3]])           # three tokens more than the sequences have
    out = torch.full_like(q, 7.0)
    o, lse = c.run(cu=np.concatenate([[0], np.cumsum(new)]), q=q, out=out)
    assert o is out and (o[sum(new):] == 7).all() and T >= sum(new)
    c.check(o, lse, [0])
    if len(new) > 2:
        k, v = c.s.tokens(2)
        r = slice(new[0], new[0] + new[2])
        compare(o[r], lse[r], attend64(c.q[r], k, v, c.kv[2] - new[2], c.scale), dtype)


@both
@every_kernel
@pytest.mark.parametrize("page_of", [0, 100, 180])      # in the first part, a middle one, the last but few
def test_an_unknown_page_in_one_part(case, page_of, dtype):
    c = Call(case, dtype)
    good, good_lse = c.run()
    near, near_lse = c.run(window=100, several=False)
    right = c.s.table[0, page_of]
    for wrong in (-1, 1 << 30):
        c.s.table[0, page_of] = wrong
        o, lse = c.run()
        # what the row's tokens see: all of them stand behind 2480
        seen = np.arange(3000 - c.new[0], 3000) >= 16 * page_of
        r, at = c.rows(0), torch.from_numpy(seen)
        assert o[r][at].isnan().all() and lse[r][at].isnan().all()
        assert torch.equal(o[r][~at], good[r][~at]) and torch.equal(lse[r][~at], good_lse[r][~at])
        rest = slice(c.new[0], None)
        assert torch.equal(o[rest], good[rest]) and torch.equal(lse[rest], good_lse[rest])
        if page_of < 100:       # before every row's window
            o, lse = c.run(window=100, several=False)
            assert torch.equal(o, near) and torch.equal(lse, near_lse)
    c.s.table[0, page_of] = right


@both
@every_kernel
def test_nan_scales_in_one_part(case, dtype):
    c = Call(case, dtype)
    good, good_lse = c.run()
    mine = c.s.table[0, 60]                 # tokens 960 .. 975, which every row sees
    G = c.H // 2
    for which in ("k_scale", "v_scale"):
        a = getattr(c.s, which)
        was = a[mine, 1]
        a[mine, 1] = np.nan                 # of key head 1
        o, lse = c.run()
        a[mine, 1] = was
        r = c.rows(0)
        assert o[r, G:].isnan().all()
        assert torch.equal(o[r, :G], good[r, :G]) and torch.equal(lse[r, :G], good_lse[r, :G])
        if which == "k_scale":
            assert lse[r, G:].isnan().all()
        else:                               # the statistics do not know the values
            k, v = c.s.tokens(0)
            _, ref, _, size = attend64(c.q[r], k, v, c.kv[0] - c.new[0], c.scale)
            assert (np.abs(lse[r].double().cpu().numpy() - ref) <= 2.0 ** -17 + 2.0 ** -19 * size).all()
        rest = slice(c.new[0], None)
        assert torch.equal(o[rest], good[rest]) and torch.equal(lse[rest], good_lse[rest])


@both
@every_kernel
def test_queries_with_nan_and_infinity_stay_in_their_rows(case, dtype):
    c = Call(case, dtype)
    good, good_lse = c.run()
    q = c.q.clone()
    q[0, 1, 3] = float("nan")
    q[c.new[0] - 1, 2, 5] = float("inf")
    o, lse = c.run(q=q)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[c.new[0] - 1, 2] = True
    assert o[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(o[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])


@both
@every_kernel
def test_rows_of_minus_infinity(case, dtype):
    """Scores below fp32's range are -inf. Row 0: all of them, which has no softmax:
    NaN. Row 1 (another head): those of most pages, so that some of its parts hold
    nothing but -inf: the other pages decide."""
    c = Call(case, dtype)
    good, good_lse = c.run()
    s = c.s
    s.keys[:, :, :, 0] = 100
    s.keys[:, :, :, 1] = 100
    kept = s.table[0, [70, 71, 150]]        # tokens 1120 .. 1151, 2400 .. 2415
    s.keys[kept, :, :, 1] = 0
    q = c.q.clone()
    q[0, 0] = q[0, 1] = 0
    q[0, 0, 0] = q[0, 1, 1] = -3e38
    o, lse = c.run(q=q)
    assert o[0, 0].isnan().all() and lse[0, 0].isnan()
    k, v = s.tokens(0)
    at = np.r_[1120:1152, 2400:2416]
    w, a = np.abs(v[at, 0]).mean(0), v[at, 0].mean(0)
    bound = (2.0 ** -8 * (w + np.abs(a)) if dtype is BF else 2.0 ** -16 * w) + 1e-30
    assert (np.abs(o[0, 1].double().cpu().numpy() - a) <= bound).all()
    assert abs(lse[0, 1].item() - np.log(48)) <= 2.0 ** -17
    rest = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    rest[0, :2] = False
    assert not o[rest].isnan().any()


@both
@every_kernel
def test_zero_tiny_and_large_scales_in_some_parts(case, dtype):
    c = Call(case, dtype)
    pages = c.s.table[0]
    c.s.v_scale[pages[10:40]] = 0.0
    c.s.v_scale[pages[40:70]] = 1e-30
    c.s.v_scale[pages[90:95]] = 1e20
    c.s.k_scale[pages[120:130]] = 0.0
    if len(c.kv) > 1:
        c.s.v_scale[c.s.table[1, :30]] = 1e-36
    o, lse = c.run()
    c.check(o, lse, range(len(c.kv)))


@both
@every_kernel
def test_the_same_bits_every_time_and_on_another_stream(case, dtype):
    c = Call(case, dtype, 128, 64)
    first = c.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(3):
            again = c.run()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("H", [4, 16, 64])
def test_graph_replays_with_rows_in_parts(H):
    """Attention captured once (one, two tiles of 16 rows, a row tile) and replayed with
    other lengths, of one part and of many, and other queries in the same buffers."""
    s = Setup([4000, 1500, 700], 2, 64, 16, 5)
    cache, lens, q = s.cache(), i32([1, 1, 1]), queries(3, H, 64, BF, 6)
    batch = s.sffn.CacheBatch(i32(s.table), lens, 4000)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.sffn.cache_attention(cache, batch, q)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = s.sffn.cache_attention(cache, batch, q, return_lse=True)
    for i, n in enumerate(([4000, 3, 700], [5, 1500, 513], [512, 512, 1], [2049, 1030, 650], [3999, 1499, 0])):
        lens.copy_(i32(n))
        q.copy_(queries(3, H, 64, BF, 7 + i))
        graph.replay()
        eager = s.sffn.cache_attention(cache, batch, q, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        for b in range(3):
            if n[b]:
                k, v = s.tokens(b)
                ref = attend64(q[b:b + 1], k[:n[b]], v[:n[b]], n[b] - 1, 0.125)
                compare(out[b:b + 1], lse[b:b + 1], ref, BF)
            else:
                assert (out[b] == 0).all() and lse[b].isneginf().all()
