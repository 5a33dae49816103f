"""Calls of the attention-side operators that take more workgroups than one grid is
given: they are launched in pieces, and give what smaller calls give."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,H,D,layout", [(600001, 32, 9, "half"),          # element by element: 19.2 million heads
                                          (17000001, 32, 8, "interleaved")])    # 16-byte accesses: 8.7 GB
def test_rotation(T, H, D, layout):
    import activation_sparse_ffn_amd as sffn
    x = torch.empty(T, H, D, dtype=BF, device="cuda")
    for part in x.split(1 << 20):
        part.normal_()
    table = sffn.rope_table(64, 8)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % 64
    w = torch.rand(D, device="cuda").to(BF)
    y, _ = sffn.qk_norm_rope(x, None, pos, table, w, layout=layout)
    for a, e in ((0, 1000), (T // 2 - 500, T // 2 + 500), (T - 1000, T)):
        z, _ = sffn.qk_norm_rope(x[a:e].contiguous(), None, pos[a:e].contiguous(), table, w, layout=layout)
        assert torch.equal(y[a:e], z)
    assert not any(p.isnan().any().item() for p in y.split(1 << 20))


def test_append():
    """4200 pages of 512 heads, keys and values: 4.3 million workgroups."""
    import activation_sparse_ffn_amd as sffn
    pages, K, D, P = 4200, 512, 64, 16
    T = pages * P - 5
    cache = sffn.KVCache.empty(pages, K, D, P)
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None]
    x = torch.empty(T, K, D, dtype=BF, device="cuda")
    for part in x.split(1 << 12):
        part.normal_()
    batch = sffn.CacheBatch(table, i32([T]), T, i32([0, T]), T)
    sffn.kv_cache_append(cache, batch, x, x)
    for a, e in ((0, 100), (T // 2, T // 2 + 100), (T - 100, T)):
        back = sffn.CacheBatch(table, i32([e]), e, i32([0, e - a]), e - a)
        k, v = sffn.kv_cache_read(cache, back, e - a)
        # half a step of a page's largest value (5 here, with room) and bf16's rounding
        assert (k.float() - x[a:e].float()).abs().max() < 5.5 / 254 + 5.5 / 256
        assert torch.equal(k, v)


def test_attention_with_a_loose_max_new():
    """2000 sequences, 64 heads, and a bound of all 40000 tokens for each of them: 20
    million workgroups, of which few have rows."""
    import activation_sparse_ffn_amd as sffn
    B, H, D, P, n = 2000, 64, 64, 16, 20
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    cache = sffn.KVCache(torch.randint(-127, 128, (B * 2, H, P, D), generator=g, device="cuda", dtype=torch.int8),
                         torch.randint(-127, 128, (B * 2, H, D, P), generator=g, device="cuda", dtype=torch.int8),
                         torch.full((B * 2, H), 0.01, device="cuda"), torch.full((B * 2, H), 0.01, device="cuda"))
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    lens = (torch.arange(B, device="cuda") % 13 + n).to(torch.int32)
    cu = torch.arange(0, n * B + 1, n, dtype=torch.int32, device="cuda")
    q = torch.randn(n * B, H, D, generator=g, device="cuda").to(BF)
    loose = sffn.cache_attention(cache, sffn.CacheBatch(table, lens, 32, cu, n * B), q)
    tight = sffn.cache_attention(cache, sffn.CacheBatch(table, lens, 32, cu, n), q)
    # both round: 2^-8 of themselves each, values are at most 1.27
    assert not loose.isnan().any() and (loose.float() - tight.float()).abs().max() < 1.27 * 2.0 ** -7
