"""The attention-side operators where no GPU is needed: refusals of the C entry
points and of the binding, and the rotary tables."""
import ctypes
import math

import pytest
import torch

import activation_sparse_ffn_amd as sffn
from activation_sparse_ffn_amd import attention as at

FAKE = 0x10000      # aligned addresses, never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


def heads(address=FAKE, st=4096, sh=128):
    return at._Heads(address, st, sh)


def rope_cfg(**kw):
    base = dict(n_q_heads=32, n_k_heads=8, head_dim=128, rot_dim=128, max_pos=100, dtype=1, layout=0, norm=1, eps=1e-6)
    base.update(kw)
    return at._RopeConfig(**base)


def cache(**kw):
    base = dict(keys=FAKE, values=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=10, kv_heads=8, page=64, head_dim=128)
    base.update(kw)
    return at._Cache(**base)


def batch(**kw):
    base = dict(block_table=FAKE, table_stride=5, kv_lens=FAKE, cu=FAKE, n_seqs=2, max_pages=5, max_new=4, max_kv=300)
    base.update(kw)
    return at._Batch(**base)


def refused(lib, status, want=sffn.SFFN_ERR_INVALID_ARG, says=""):
    assert status == want, (status, lib.sparse_ffn_last_error())
    assert says.encode() in lib.sparse_ffn_last_error(), lib.sparse_ffn_last_error()


@pytest.mark.parametrize("bad,says", [
    (dict(n_q_heads=0), "n_q_heads"), (dict(n_k_heads=-1), "n_k_heads"), (dict(head_dim=0), "head_dim"),
    (dict(head_dim=513), "head_dim"), (dict(rot_dim=3), "rot_dim"), (dict(rot_dim=130), "rot_dim"),
    (dict(rot_dim=-2), "rot_dim"), (dict(max_pos=0), "max_pos"), (dict(dtype=2), "dtype"), (dict(layout=2), "layout"),
    (dict(norm=2), "norm"), (dict(eps=0.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(n_q_heads=1 << 20), "n_q_heads"),
])
def test_rope_configs(lib, bad, says):
    h, c = heads(), rope_cfg(**bad)
    refused(lib, lib.qk_norm_rope(c, h, h, FAKE, FAKE, None, None, 4, h, h, None), says=says)
    refused(lib, lib.qk_norm_rope_backward(c, h, h, h, h, FAKE, FAKE, None, None, 4, h, h, None, None, None, 0, None),
            says=says)
    assert lib.qk_norm_rope_backward_workspace_size(c, 4) == 0


def test_rope_arguments(lib):
    h, c = heads(), rope_cfg()

    def call(q=h, k=h, pos=FAKE, table=FAKE, w=None, T=4, q_out=h, k_out=h):
        return lib.qk_norm_rope(c, q, k, pos, table, w, None, T, q_out, k_out, None)

    refused(lib, call(T=-1), says="T must")
    refused(lib, call(T=1 << 40), sffn.SFFN_ERR_UNSUPPORTED, "too large")
    refused(lib, call(q=None), says="q is null")
    refused(lib, call(k=heads(0)), says="k is null")
    refused(lib, call(q_out=None), says="q_out is null")
    refused(lib, call(pos=None), says="positions")
    refused(lib, call(table=FAKE + 2), says="aligned")
    refused(lib, call(w=FAKE + 1), says="weights")
    refused(lib, call(q=heads(FAKE + 1)), says="aligned")
    refused(lib, call(q=heads(st=-1)), says="strides")
    refused(lib, call(q=heads(st=1 << 50)), says="strides")
    refused(lib, call(q_out=heads(st=0)), says="overlaps")
    refused(lib, call(q_out=heads(st=4096, sh=64)), says="overlaps")
    refused(lib, call(k_out=heads(st=128, sh=256)), says="overlaps")        # four tokens need 512 a head
    assert call(T=0, q=None, k=None) == sffn.SFFN_OK
    b = lib.qk_norm_rope_backward
    refused(lib, b(c, h, h, h, h, FAKE, FAKE, FAKE, FAKE, 4, h, h, FAKE, FAKE, None, 0, None), says="workspace is null")
    refused(lib, b(c, h, h, h, h, FAKE, FAKE, FAKE, FAKE, 4, h, h, FAKE, FAKE, FAKE + 16, 1 << 30, None), says="256")
    refused(lib, b(c, h, h, h, h, FAKE, FAKE, FAKE, FAKE, 4, h, h, FAKE, FAKE, FAKE, 16, None),
            sffn.SFFN_ERR_WORKSPACE, "needed")
    refused(lib, b(c, None, h, h, h, FAKE, FAKE, FAKE, FAKE, 4, h, h, FAKE, FAKE, FAKE, 1 << 30, None), says="q is null")
    refused(lib, b(c, h, h, h, h, FAKE, FAKE, FAKE, FAKE, 4, h, h, FAKE + 2, FAKE, FAKE, 1 << 30, None), says="aligned")
    assert lib.qk_norm_rope_backward_workspace_size(c, 0) == 0
    assert lib.qk_norm_rope_backward_workspace_size(c, 4) > 0
    assert lib.qk_norm_rope_backward_workspace_size(rope_cfg(norm=0), 4) == 0


BAD_CACHE = [(dict(page=24), sffn.SFFN_ERR_UNSUPPORTED, "page"), (dict(head_dim=96), sffn.SFFN_ERR_UNSUPPORTED, "head_dim"),
             (dict(kv_heads=0), 1, "kv_heads"), (dict(n_pages=0), 1, "n_pages"), (dict(n_pages=1 << 31), 1, "n_pages"),
             (dict(keys=None), 1, "keys"), (dict(values=FAKE + 8), 1, "aligned"), (dict(v_scale=None), 1, "v_scale")]
BAD_BATCH = [(dict(n_seqs=-1), 1, "negative"), (dict(max_new=-1), 1, "negative"), (dict(table_stride=4), 1, "table_stride"),
             (dict(table_stride=-5), 1, "table_stride"), (dict(max_pages=1 << 28, table_stride=1 << 28), 2, "max_pages"),
             (dict(max_pages=0), 1, "max_pages"), (dict(kv_lens=None), 1, "kv_lens"), (dict(block_table=None), 1, "block_table"),
             (dict(cu=FAKE + 2), 1, "aligned"), (dict(cu=None), 1, "without cu"), (dict(cu=None, n_seqs=4, max_new=0), 1, "max_new")]


@pytest.mark.parametrize("c,b,want,says", [(c, {}, w, s) for c, w, s in BAD_CACHE] + [({}, b, w, s) for b, w, s in BAD_BATCH])
def test_caches_and_batches(lib, c, b, want, says):
    h, C, B = heads(), cache(**c), batch(**b)
    refused(lib, lib.kv_cache_append(C, B, h, h, 1, 4, None), want, says)
    refused(lib, lib.kv_cache_read(C, B, h, h, 1, 4, None), want, says)
    refused(lib, lib.cache_attention(C, B, h, 32, 1, 4, 0.1, 0, h, None, FAKE, 1 << 40, None), want, says)


def test_cache_arguments(lib):
    h, C, B = heads(), cache(), batch()
    for f in (lib.kv_cache_append, lib.kv_cache_read):
        refused(lib, f(C, B, h, h, 2, 4, None), says="dtype")
        refused(lib, f(C, B, h, h, 1, -4, None), says="T must")
        refused(lib, f(C, B, h, h, 1, 1 << 40, None), sffn.SFFN_ERR_UNSUPPORTED, "too large")
        refused(lib, f(C, B, None, h, 1, 4, None), says="k is null")
        refused(lib, f(C, B, h, heads(st=4097), 1, 4, None), says="16-byte")
        refused(lib, f(None, B, h, h, 1, 4, None), says="null")
        assert f(C, B, None, None, 1, 0, None) == sffn.SFFN_OK
    refused(lib, lib.kv_cache_read(C, B, heads(st=0), h, 1, 4, None), says="overlaps")

    def attend(q=h, n=32, dt=1, T=4, scale=0.1, window=0, out=h, lse=None, ws=FAKE, size=1 << 40, b=B):
        return lib.cache_attention(C, b, q, n, dt, T, scale, window, out, lse, ws, size, None)

    refused(lib, attend(n=30), says="multiple")
    refused(lib, attend(n=0), says="multiple")
    refused(lib, attend(window=-1), says="window")
    refused(lib, attend(scale=math.inf), says="scale")
    refused(lib, attend(dt=7), says="dtype")
    refused(lib, attend(q=heads(FAKE + 2)), says="16-byte")
    refused(lib, attend(out=heads(sh=0)), says="overlaps")
    refused(lib, attend(lse=FAKE + 1), says="lse")
    long = batch(max_kv=30000)
    need = lib.cache_attention_workspace_size(C, long, 32, 1, 0, 4)
    assert need > 0
    refused(lib, attend(b=long, ws=None), says="workspace is null")
    refused(lib, attend(b=long, ws=FAKE + 16), says="256")
    refused(lib, attend(b=long, size=need - 1), sffn.SFFN_ERR_WORKSPACE, "needed")
    refused(lib, attend(b=batch(n_seqs=1 << 20, max_pages=1 << 16, table_stride=1 << 16)), sffn.SFFN_ERR_UNSUPPORTED, "too many")
    assert attend(T=0, q=None, out=None) == sffn.SFFN_OK
    assert lib.cache_attention_workspace_size(C, batch(max_kv=100), 32, 1, 0, 4) == 0       # one part
    assert lib.cache_attention_workspace_size(C, long, 30, 1, 0, 4) == 0
    # more keys, more parts; a window bounds them
    sizes = [lib.cache_attention_workspace_size(C, batch(max_kv=n), 32, 1, 0, 4) for n in (1000, 5000, 30000)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[-1]
    assert lib.cache_attention_workspace_size(C, long, 32, 1, 500, 4) < need


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        sffn.qk_norm_rope(x, None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        sffn.KVCache(torch.zeros(1, 1, 16, 64, dtype=torch.int8), None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        sffn.CacheBatch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1)
    with pytest.raises(TypeError):
        sffn.qk_norm_rope(None, None, None, None)


def test_rope_table_closed_forms():
    t = sffn.rope_table(10, 4, base=100.0, device="cpu")
    assert t.shape == (10, 4) and t.dtype == torch.float32
    for p in range(10):
        for i, f in enumerate((1.0, 0.1)):
            assert abs(t[p, i].item() - math.cos(p * f)) < 1e-7 and abs(t[p, 2 + i].item() - math.sin(p * f)) < 1e-7
    # by_parts: the ramp from 1 to 32 turns in the trained context
    base, trained, factor = 10000.0, 4096, 8.0
    t = sffn.rope_table(2, 128, base=base, scaling="by_parts", factor=factor, original_max_pos=trained, device="cpu")
    amp = 1 + 0.1 * math.log(factor)
    for i in range(64):
        f = base ** (-2 * i / 128)
        keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - 1) / 31))
        f = f * keep + f / factor * (1 - keep)
        assert abs(t[1, i].item() - amp * math.cos(f)) < 1e-6


@pytest.mark.parametrize("kw", [dict(max_pos=0), dict(rot_dim=5), dict(rot_dim=0), dict(scaling="other"), dict(factor=0.0),
                                dict(base=-1.0), dict(scaling="by_parts")])
def test_rope_table_refusals(kw):
    args = dict(max_pos=8, rot_dim=4, device="cpu")
    args.update(kw)
    with pytest.raises(ValueError):
        sffn.rope_table(**args)


def test_struct_sizes_match_the_header():
    """Four structs cross the boundary by pointer; their layouts are the C ones."""
    assert ctypes.sizeof(at._Heads) == 24 and ctypes.sizeof(at._RopeConfig) == 36
    assert ctypes.sizeof(at._Cache) == 56 and ctypes.sizeof(at._Batch) == 48
