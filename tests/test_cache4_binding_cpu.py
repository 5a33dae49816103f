"""The 4-bit cache where no GPU is needed: refusals of the C entry points and of the binding,
and the device that a call is launched on."""
import contextlib

import pytest
import torch

import activation_sparse_ffn_amd as sffn
from activation_sparse_ffn_amd import attention as at
from tests.test_attention_binding_cpu import FAKE, batch, heads, refused

INVALID, UNSUPPORTED = sffn.SFFN_ERR_INVALID_ARG, sffn.SFFN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


def cache(**kw):
    base = dict(keys=FAKE, values=FAKE, k_exp=FAKE, v_scale=FAKE, n_pages=10, kv_heads=8, page=64, head_dim=128)
    base.update(kw)
    return at._Cache4(**base)


def calls(lib, c, b, T=8, k=None, q=None, slots=None):
    """The three calls over a cache and a batch; every one is refused."""
    k, q = k or heads(st=1024), q or heads()
    yield lib.kv_cache4_append(c, b, slots, k, k, 1, T, None)
    yield lib.kv_cache4_read(c, b, k, k, 1, T, None)
    yield lib.cache4_attention(c, b, q, 32, 1, T, 0.1, 0, q, None, FAKE, 1 << 40, None)


@pytest.mark.parametrize("bad,says,want", [
    (dict(keys=None), "keys is null", INVALID), (dict(values=None), "values is null", INVALID),
    (dict(k_exp=None), "k_exp is null", INVALID), (dict(v_scale=None), "v_scale is null", INVALID),
    (dict(keys=FAKE + 8), "keys is not 16-byte", INVALID), (dict(k_exp=FAKE + 4), "k_exp is not 16-byte", INVALID),
    (dict(n_pages=0), "n_pages", INVALID), (dict(n_pages=1 << 31), "n_pages", INVALID),
    (dict(kv_heads=0), "kv_heads", INVALID), (dict(page=8), "page must", UNSUPPORTED),
    (dict(page=256), "page must", UNSUPPORTED), (dict(head_dim=32), "head_dim", UNSUPPORTED),
    (dict(head_dim=512), "head_dim", UNSUPPORTED),
])
def test_caches(lib, bad, says, want):
    for st in calls(lib, cache(**bad), batch()):
        refused(lib, st, want, says)


@pytest.mark.parametrize("bad,says,want", [
    (dict(n_seqs=-1), "n_seqs", INVALID), (dict(max_new=-1), "max_new", INVALID), (dict(max_kv=-1), "max_kv", INVALID),
    (dict(max_pages=-1), "max_pages", INVALID), (dict(max_pages=0), "max_pages", INVALID),
    (dict(table_stride=4), "table_stride", INVALID),
    (dict(max_pages=1 << 25, table_stride=1 << 25), "too many", UNSUPPORTED),
    (dict(kv_lens=None), "block_table and kv_lens", INVALID), (dict(block_table=None), "block_table and", INVALID),
    (dict(block_table=FAKE + 2), "4-byte aligned", INVALID), (dict(cu=None), "without cu", INVALID),
])
def test_batches(lib, bad, says, want):
    for st in calls(lib, cache(), batch(**bad)):
        refused(lib, st, want, says)


def test_arguments(lib):
    c, b, k, q = cache(), batch(), heads(st=1024), heads()
    for st in calls(lib, None, b):
        refused(lib, st, says="must not be null")
    for st in calls(lib, c, b, T=-1):
        refused(lib, st, says="T must")
    for st in calls(lib, c, b, T=(1 << 28) + 1):
        refused(lib, st, UNSUPPORTED, "too large")
    for bad, says in ((heads(0), "is null"), (heads(FAKE + 2), "16-byte"), (heads(st=1028), "16-byte"),
                      (heads(st=-8), "strides"), (heads(sh=1 << 50), "strides")):
        for st in calls(lib, c, b, k=bad, q=bad):
            refused(lib, st, says=says)
    refused(lib, lib.kv_cache4_read(c, b, heads(st=1024, sh=64), k, 1, 8, None), says="overlaps")

    def append(slots=FAKE, cache=c, T=8, dtype=1, k=k):
        return lib.kv_cache4_append(cache, None, slots, k, k, dtype, T, None)

    refused(lib, append(slots=None), says="must not be null")
    refused(lib, append(slots=FAKE + 4), says="slots must be 8-byte")
    refused(lib, append(T=-1), says="T must")
    refused(lib, append(T=1 << 31), says="T must")
    refused(lib, append(T=(1 << 28) + 1), UNSUPPORTED, "too large")
    refused(lib, append(dtype=7), says="dtype")
    refused(lib, append(cache=cache(kv_heads=1 << 17)), says="kv_heads")

    def attend(heads=32, T=8, scale=0.1, window=0, out=q, lse=None, ws=FAKE, size=1 << 40, dtype=1, b=b):
        return lib.cache4_attention(c, b, q, heads, dtype, T, scale, window, out, lse, ws, size, None)

    refused(lib, attend(heads=33), says="n_q_heads")
    refused(lib, attend(heads=0), says="n_q_heads")
    refused(lib, attend(window=-1), says="window")
    refused(lib, attend(scale=float("inf")), says="scale")
    refused(lib, attend(scale=float("nan")), says="scale")
    refused(lib, attend(dtype=3), says="dtype")
    refused(lib, attend(out=None), says="out is null")
    refused(lib, attend(out=heads(st=4096, sh=64)), says="overlaps")
    refused(lib, attend(lse=FAKE + 2), says="lse")
    refused(lib, attend(T=1 << 28), UNSUPPORTED, "too large")
    # a batch whose parts need room
    long = batch(max_pages=1000, table_stride=1000, max_kv=60000)
    need = lib.cache4_attention_workspace_size(c, long, 32, 1, 0, 8)
    assert 0 < need <= 256 << 20
    refused(lib, attend(b=long, ws=None), says="workspace is null")
    refused(lib, attend(b=long, ws=FAKE + 16), says="256-byte")
    refused(lib, attend(b=long, size=need - 1), sffn.SFFN_ERR_WORKSPACE, "needed")
    assert lib.cache4_attention_workspace_size(cache(page=8), long, 32, 1, 0, 8) == 0
    assert lib.cache4_attention_workspace_size(c, long, 33, 1, 0, 8) == 0
    assert lib.cache4_attention_workspace_size(c, long, 32, 9, 0, 8) == 0


def test_nothing_to_do_needs_no_buffers(lib):
    empty = cache(keys=None, values=None, k_exp=None, v_scale=None)
    for b in (batch(block_table=None, kv_lens=None, n_seqs=0), batch(max_new=0)):
        assert lib.kv_cache4_append(empty, b, None, None, None, 1, 8, None) == 0
        assert lib.kv_cache4_read(empty, b, None, None, 1, 8, None) == 0
        assert lib.cache4_attention(empty, b, None, 32, 1, 8, 0.1, 0, None, None, None, 0, None) == 0
    assert lib.kv_cache4_append(empty, None, FAKE, None, None, 1, 0, None) == 0


def test_tensors_are_checked_before_their_addresses_are_taken():
    u8 = dict(dtype=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        sffn.KVCache4(torch.zeros(2, 2, 16, 32, **u8), torch.zeros(2, 2, 16, 32, **u8), torch.zeros(2, 2, 16, 2, **u8),
                      torch.zeros(2, 2, 16))
    with pytest.raises(ValueError, match="on the GPU"):
        sffn.KVCache4(torch.zeros(2, 2, **u8), *[torch.zeros(1)] * 3)


@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_for_the_launch(monkeypatch, current):
    """On the default stream a launch goes to the current device."""
    entered, handed = [], []

    @contextlib.contextmanager
    def device(d):
        entered.append(d.index)
        yield

    monkeypatch.setattr(sffn, "_current_device", lambda: current)
    monkeypatch.setattr(sffn, "_raw_stream", lambda i: 1000 + i)
    monkeypatch.setattr(torch.cuda, "device", device)
    sffn._run(None, torch.device("cuda", 1), lambda *a: handed.append(a) or 0, "x")
    assert handed == [("x", 1001)] and entered == ([] if current == 1 else [1])
