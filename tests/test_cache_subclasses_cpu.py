"""A cache of a class of the user's own, derived from one of the package's, goes where its base
goes. Without a GPU: the library and the launch are faked, and which entry points the binding
calls is recorded."""
from types import SimpleNamespace

import pytest
import torch

import activation_sparse_ffn_amd as sffn
from activation_sparse_ffn_amd import attention as at


class Library:
    """Every entry point is its own name; sizes are 0."""

    def __getattr__(self, name):
        return (lambda *a: 0) if name.endswith("workspace_size") else name


@pytest.mark.parametrize("base,names", [(sffn.KVCache, ["kv_cache_append", "kv_cache_read", "cache_attention"]),
                                        (sffn.KVCache4, ["kv_cache4_append", "kv_cache4_read", "cache4_attention"])])
def test_the_entry_points_of_a_derived_cache(monkeypatch, base, names):
    called = []
    monkeypatch.setattr(at, "load_library", Library)
    monkeypatch.setattr(at, "_run", lambda lib, device, call, *args: called.append(call))
    monkeypatch.setattr(at, "_heads", lambda t, *a: None)
    cpu = torch.device("cpu")
    kv, q = torch.zeros(3, 2, 64), torch.zeros(3, 4, 64)
    for kind in (base, type("Named", (base,), {})):
        cache = object.__new__(kind)
        cache.device, cache.kv_heads, cache.page, cache.head_dim, cache._c = cpu, 2, 16, 64, None
        batch = SimpleNamespace(device=cpu, slots=None, _c=None)
        called.clear()
        at.kv_cache_append(cache, batch, kv, kv)
        at.kv_cache_read(cache, batch, 3, torch.float32)
        at.cache_attention(cache, batch, q)
        assert called == names, kind
