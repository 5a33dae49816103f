"""Calls whose tokens all lie behind the last sequence, as the steps of a captured graph that
no sequence takes part in: nothing is read, written or stored, over either cache and in every
kernel's range of sizes; the next replay with tokens is the eager call's."""
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(bits, D, B):
    """A cache with 200 tokens in each of B sequences, and their table."""
    import activation_sparse_ffn_amd as sffn
    cache = (sffn.KVCache4 if bits == 4 else sffn.KVCache).empty(4 * B, 2, D, 64)
    for t in (cache.keys, cache.values):
        t.zero_()
    table = torch.arange(4 * B, dtype=torch.int32, device="cuda").view(B, 4)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(200 * B, 2, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    cu = i32([200 * b for b in range(B + 1)])
    sffn.kv_cache_append(cache, sffn.CacheBatch(table, i32([200] * B), 200, cu, 200), k, v)
    return cache, table


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
# rows of a tile of 16, of two, of row tiles; one sequence, a few, more than a wave has lanes
@pytest.mark.parametrize("B,max_new,T,max_kv", [(1, 1, 3, 200), (1, 40, 40, 9000), (3, 1, 3, 200), (3, 4, 9, 60000),
                                                (3, 7, 21, 200), (3, 60, 70, 9000), (70, 1, 70, 9000), (70, 30, 90, 200)])
def test_no_sequence_has_new_tokens(B, max_new, T, max_kv, D, dtype, bits):
    import activation_sparse_ffn_amd as sffn
    cache, table = filled(bits, D, B)
    names = ("keys", "values", "k_exp", "v_scale") if bits == 4 else ("keys", "values", "k_scale", "v_scale")
    held = [getattr(cache, n) for n in names]
    before = [t.clone() for t in held]
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(T, 8, D, generator=g, device="cuda").to(dtype)
    kv = torch.randn(T, 2, D, generator=g, device="cuda").to(dtype)
    for window in (0, 50):
        for first in (0, T):        # where the empty sequences stand
            batch = sffn.CacheBatch(table, i32([200] * B), max_kv, i32([first] * (B + 1)), max_new)
            out = torch.full((T, 8, D), 3.0, dtype=dtype, device="cuda")
            sffn.kv_cache_append(cache, batch, kv, kv)
            o, _ = sffn.cache_attention(cache, batch, q, window=window, out=out, return_lse=True)
            k, v = sffn.kv_cache_read(cache, batch, T, dtype, k=kv.clone(), v=kv.clone())
            torch.cuda.synchronize()
            assert o is out and (out == 3).all() and torch.equal(k, kv) and torch.equal(v, kv)
    for a, b in zip(before, held):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("most", [1, 5, 40])
def test_a_captured_call_with_and_without_tokens(most, bits):
    import activation_sparse_ffn_amd as sffn
    B, D = 3, 128
    cache, table = filled(bits, D, B)
    T = B * most
    q = torch.randn(T, 8, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    cu, lens, out = i32([0] * (B + 1)), i32([200] * B), torch.zeros_like(q)
    batch = sffn.CacheBatch(table, lens, 256, cu, most)
    sffn.cache_attention(cache, batch, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sffn.cache_attention(cache, batch, q, out=out)
    for offsets in ([0, 0, 0, 0], [0, most, most, 2 * most], [0, 0, 0, 0], [0, 1, 1, 1], [0, most, 2 * most, 3 * most]):
        cu.copy_(i32(offsets))
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = sffn.cache_attention(cache, batch, q, out=torch.full_like(q, 3))
        assert torch.equal(out, want) and (out[offsets[-1]:] == 3).all()
        assert torch.isfinite(out.float()).all()
