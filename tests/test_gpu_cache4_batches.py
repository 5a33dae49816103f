"""Batches of the 4-bit cache whose tokens are not all stored or not all there: the same
whether slots are given or looked up. Whole numbers and copies: everything is equal."""
import numpy as np
import pytest
import torch

from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def buffers(cache):
    return [t.view(torch.uint8) for t in (cache.keys, cache.values, cache.k_exp, cache.v_scale)]


def unused(n_pages, heads, dim, page):
    """A cache of which every byte is 77."""
    import activation_sparse_ffn_amd as sffn
    cache = sffn.KVCache4.empty(n_pages, heads, dim, page)
    for t in buffers(cache):
        t.fill_(77)
    return cache


def normal(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,most,max_new", [(1, 9, 4), (1, 9, 9), (3, 6, 1), (8, 5, 2), (9, 5, 3), (33, 4, 2), (70, 9, 3),
                                            (600, 5, 4), (3000, 3, 1)])
def test_an_append_by_slots_stores_what_one_by_tables_stores(B, most, max_new, D):
    """page_plan gives every token a slot; those beyond max_new are stored by neither."""
    import activation_sparse_ffn_amd as sffn
    r = np.random.default_rng(B + D)
    new = r.integers(0, most + 1, B)
    new[r.integers(B)] = most
    T = int(new.sum())
    free, n_free = sffn.free_pages(2 * B)
    table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    held = r.integers(0, 20, B)
    first = sffn.page_plan(table, i32([0] * B), i32(held), free, n_free, 16, int(held.sum()))
    plan = sffn.page_plan(table, first.kv_lens, i32(new), free, first.n_free, 16, T + 3)
    k, v = normal(T + 3, 3, D, seed=1), normal(T + 3, 3, D, seed=2)
    caches = [unused(2 * B, 3, D, 16) for _ in range(2)]
    for cache, slots in zip(caches, (None, plan.slots)):
        batch = sffn.CacheBatch(table, plan.kv_lens, 40, plan.cu, max_new, slots=slots)
        sffn.kv_cache_append(cache, batch, k, v)
    for a, b in zip(*map(buffers, caches)):
        assert torch.equal(a, b)
    # what is stored: the tokens with a slot among their sequence's first max_new
    cu, slots = plan.cu.cpu().numpy(), plan.slots.cpu().numpy()
    want = {int(slots[t]) for b in range(B) for t in range(cu[b], cu[b + 1]) if t - cu[b] < max_new and slots[t] >= 0}
    scales = caches[1].v_scale.view(torch.int32)[:, 0].flatten().cpu().numpy()
    assert set(np.flatnonzero(scales != 0x4d4d4d4d).tolist()) == want


def test_slots_of_tokens_of_no_sequence():
    """Of the batch only max_new tells a token with a slot from one that is not stored."""
    import activation_sparse_ffn_amd as sffn
    k = normal(8, 2, 64)
    everything = list(range(8))
    for cu, max_new, stored in (([2, 4, 7], 8, everything), ([2, 4, 7], 2, [0, 1, 2, 3, 4, 5]), ([0, 0, 0], 8, everything),
                                ([8, 8, 8], 1, everything), ([0, 5, 8], 3, [0, 1, 2, 5, 6, 7]), ([0, 4, 8], 0, []),
                                (None, 1, everything)):
        cache = unused(2, 2, 64, 16)
        batch = sffn.CacheBatch(i32([[0], [1]]), i32([9, 9]), 9, None if cu is None else i32(cu), max_new,
                                slots=torch.arange(3, 11, device="cuda"))
        sffn.kv_cache_append(cache, batch, k, k)
        scales = cache.v_scale.view(torch.int32)[0, 0].cpu().numpy()
        assert (np.flatnonzero(scales != 0x4d4d4d4d) - 3).tolist() == stored
    # no sequences at all
    cache = unused(2, 2, 64, 16)
    batch = sffn.CacheBatch(torch.empty(0, 1, dtype=torch.int32, device="cuda"), i32([]), 9, i32([0]), 1,
                            slots=torch.arange(8, device="cuda"))
    sffn.kv_cache_append(cache, batch, k, k)
    assert (cache.v_scale.view(torch.int32)[0, 0] != 0x4d4d4d4d).sum() == 8
