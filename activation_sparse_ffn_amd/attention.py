"""The attention-side operators of a decoder layer that stand next to the sparse
FFN: norms of q and k for each head with the rotary positions, a paged cache
that holds keys and values in 8 bits or in 4, and attention over it.

    table = rope_table(32768, 128)
    q, k = qk_norm_rope(q, k, positions, table, q_weight=w_q, k_weight=w_k)
    cache = KVCache.empty(n_pages, kv_heads, head_dim)      # or KVCache4.empty
    batch = CacheBatch(block_table, kv_lens, max_kv, cu, max_new)
    kv_cache_append(cache, batch, k, v)
    o = cache_attention(cache, batch, q)

A thin ctypes binding of include/sparse_ffn_attention.h: the arithmetic runs in
the library's HIP kernels, asynchronously on torch's current stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from . import SFFN_BF16, SFFN_F32, _check, _need_buffer, _ptr, _run, _stream, load_library

__all__ = ["rope_table", "qk_norm_rope", "qk_norm_rope_backward", "KVCache", "KVCache4", "CacheBatch",
           "kv_cache_append", "kv_cache_read", "cache_attention"]

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = (None, "linear", "ntk", "by_parts")
_DTYPES = {torch.bfloat16: SFFN_BF16, torch.float32: SFFN_F32}
_INT32_MAX = 2 ** 31 - 1
_empty_strided = torch.empty_strided


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class _RopeConfig(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("max_pos", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("layout", ctypes.c_int), ("norm", ctypes.c_int32), ("eps", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("keys", ctypes.c_void_p), ("values", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Cache4(ctypes.Structure):
    _fields_ = [("keys", ctypes.c_void_p), ("values", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("page", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("kv_lens", ctypes.c_void_p),
                ("cu", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_kv", ctypes.c_int32)]


EXPORTED_SYMBOLS = ("qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_backward_workspace_size",
                    "kv_cache_append", "kv_cache_read", "cache_attention", "cache_attention_workspace_size",
                    "kv_cache4_append", "kv_cache4_read", "cache4_attention", "cache4_attention_workspace_size")


def declare(lib):
    """The signatures of include/sparse_ffn_attention.h."""
    P, S, I64, I32, F, st = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                             ctypes.c_int)
    H, R, C, B = (ctypes.POINTER(x) for x in (_Heads, _RopeConfig, _Cache, _Batch))
    lib.qk_norm_rope.argtypes = [R, H, H, P, P, P, P, I64, H, H, P]
    lib.qk_norm_rope.restype = st
    lib.qk_norm_rope_backward_workspace_size.argtypes = [R, I64]
    lib.qk_norm_rope_backward_workspace_size.restype = S
    lib.qk_norm_rope_backward.argtypes = [R, H, H, H, H, P, P, P, P, I64, H, H, P, P, P, S, P]
    lib.qk_norm_rope_backward.restype = st
    for f in (lib.kv_cache_append, lib.kv_cache_read):
        f.argtypes = [C, B, H, H, st, I64, P]
        f.restype = st
    lib.cache_attention_workspace_size.argtypes = [C, B, I32, st, I32, I64]
    lib.cache_attention_workspace_size.restype = S
    lib.cache_attention.argtypes = [C, B, H, I32, st, I64, F, I32, H, P, P, S, P]
    lib.cache_attention.restype = st
    C4 = ctypes.POINTER(_Cache4)
    lib.kv_cache4_append.argtypes = [C4, B, P, H, H, st, I64, P]
    lib.kv_cache4_append.restype = st
    lib.kv_cache4_read.argtypes = [C4, B, H, H, st, I64, P]
    lib.kv_cache4_read.restype = st
    lib.cache4_attention_workspace_size.argtypes = [C4, B, I32, st, I32, I64]
    lib.cache4_attention_workspace_size.restype = S
    lib.cache4_attention.argtypes = [C4, B, H, I32, st, I64, F, I32, H, P, P, S, P]
    lib.cache4_attention.restype = st


# ---------------------------------------------------------------------------
# argument checks
#
# A call on one token is bound by what the host does before the launch (about 3
# us of it are the launch), so the checks that pass are written to be short; the
# messages are made only for those that do not.
# ---------------------------------------------------------------------------

def _heads(t: Optional[torch.Tensor], name: str, shape=None, dtype=None, device=None):
    """A [T, heads, head_dim] view on the GPU as the library takes it. With a shape,
    dtype is one of _DTYPES and device a GPU."""
    if shape is None or type(t) is not torch.Tensor or t.shape != shape or t.dtype is not dtype or t.device != device:
        _check_heads(t, name, shape, dtype, device)
        shape = t.shape
    T, H, D = shape
    st, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # a dimension of one element may carry any stride
    if H == 1:
        sh = D
    return _Heads(t.data_ptr(), st if T > 1 else sh * H, sh)


def _check_heads(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {tuple(shape) if shape else '[T, heads, head_dim]'} "
                         f"(got {tuple(t.shape)})")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype or 'bfloat16 or float32'} (got {t.dtype})")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'the GPU'} (got {t.device})")


def _new(shape, dtype, device):
    """A new contiguous [T, heads, head_dim] tensor and what the library takes of it.
    (empty_strided is the shortest of torch's ways to one.)"""
    _, H, D = shape
    t = _empty_strided(shape, (H * D, D, 1), dtype=dtype, device=device)
    return t, _Heads(t.data_ptr(), H * D, D)


def _int32(n: int) -> int:
    """A count or bound as the library's int32 (ctypes would take its low bits): past 31
    bits it bounds nothing, below zero it is refused there."""
    return n if 0 <= n <= _INT32_MAX else _INT32_MAX if n > 0 else -1


def _vector(n, dtype, device):
    return _empty_strided((n,), (1,), dtype=dtype, device=device)


def _address(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The address of a contiguous tensor (shape None: any)."""
    if type(t) is not torch.Tensor or t.dtype is not dtype or t.device != device or not t.is_contiguous() \
            or (shape is not None and t.shape != shape):
        _need_buffer(t, name, shape, dtype, device)
    return t.data_ptr()


# ---------------------------------------------------------------------------
# head norms and rotary positions
# ---------------------------------------------------------------------------

def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original_max_pos: Optional[int] = None, device="cuda") -> torch.Tensor:
    """cos | sin of every position and pair, fp32 [max_pos, rot_dim]: made once
    for a model, in 64 bits. Pair i turns by pos * base^(-2i / rot_dim); for
    contexts `factor` times the trained one (original_max_pos tokens)

      "linear"    positions are divided by factor;
      "ntk"       base grows by factor^(rot_dim / (rot_dim - 2)), so that the
                  slowest pair turns 1 / factor as fast and the fastest as before;
      "by_parts"  pairs that turn less than once in the trained context are
                  divided by factor, those that turn 32 times or more are kept,
                  a ramp between; cos and sin are scaled by 1 + 0.1 ln factor.
    """
    if max_pos < 1 or rot_dim < 2 or rot_dim % 2:
        raise ValueError("max_pos must be positive and rot_dim a positive even number")
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {ROPE_SCALINGS}")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    exponent = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** -exponent
    amplitude = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if not original_max_pos or original_max_pos < 1:
            raise ValueError("by_parts needs original_max_pos, the trained context")
        turns = original_max_pos * freq / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        amplitude = 1 + 0.1 * math.log(factor) if factor > 1 else 1.0
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], 1) * amplitude).float().to(device)


@functools.lru_cache(maxsize=256)
def _rope_config(n_q, n_k, dim, rot, max_pos, dtype, layout, norm, eps):
    """The library's config, a constant of its arguments."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    return _RopeConfig(n_q, n_k, dim, rot, max_pos, _DTYPES[dtype], ROPE_LAYOUTS[layout], norm, eps)


def _rope_call(x, other, positions, table, q_weight, k_weight, norm, eps, layout):
    """The config and shared pointers of a call on q (or its gradient) `x` and
    k `other` (or None)."""
    T, n_q, D = x.shape
    dev, dtype = x.device, x.dtype
    wq = None if q_weight is None else _address(q_weight, "q_weight", (D,), dtype, dev)
    wk = None if k_weight is None else _address(k_weight, "k_weight", (D,), dtype, dev)
    weighted = wq is not None or wk is not None
    if norm is None:
        norm = weighted
    elif weighted and not norm:
        raise ValueError("weights are given but norm is False")
    rot = max_pos = 0
    pos = tab = None
    if table is not None:
        if table.dim() != 2:
            raise ValueError("table must be [max_pos, rot_dim] float32")
        max_pos, rot = table.shape
        tab = _address(table, "table", None, torch.float32, dev)
        pos = _address(positions, "positions", (T,), torch.int32, dev)
    cfg = _rope_config(n_q, 0 if other is None else other.shape[1], D, rot, max_pos, dtype, layout, int(norm), eps)
    return cfg, pos, tab, wq, wk


def _like_k(k, q):
    """The shape k must have: q's with its own count of heads."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [T, heads, head_dim]")
    T, _, D = q.shape
    return (T, k.shape[1], D)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                 table: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, norm: Optional[bool] = None, eps: float = 1e-6,
                 layout: str = "half", q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """RMS norm of every head of q [T, H, D] and k [T, K, D] (views with any
    token and head strides), then the rotation of its first table.shape[1]
    elements by positions [T] int32.

    norm: None takes it from whether weights are given; True without weights
    norms alone, False rotates alone. table None: no rotation. layout: "half"
    pairs (i, i + rot / 2), "interleaved" pairs (2i, 2i + 1). k may be None.
    q_out, k_out may be q and k themselves. Returns (q_out, k_out). A position
    outside the table gives NaN rows."""
    lib = load_library()
    hq = _heads(q, "q")
    dtype, dev = q.dtype, q.device
    hk = None if k is None else _heads(k, "k", _like_k(k, q), dtype, dev)
    cfg, pos, tab, wq, wk = _rope_call(q, k, positions, table, q_weight, k_weight, norm, eps, layout)
    hko = None
    if q_out is None:
        q_out, ho = _new(q.shape, dtype, dev)
    else:
        ho = _heads(q_out, "q_out", q.shape, dtype, dev)
    if k is not None:
        if k_out is None:
            k_out, hko = _new(k.shape, dtype, dev)
        else:
            hko = _heads(k_out, "k_out", k.shape, dtype, dev)
    _check(lib, lib.qk_norm_rope(cfg, hq, hk, pos, tab, wq, wk, q.shape[0], ho, hko, _stream(dev)))
    return q_out, k_out


def qk_norm_rope_backward(q: Optional[torch.Tensor], k: Optional[torch.Tensor], g_q: torch.Tensor,
                          g_k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                          table: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                          k_weight: Optional[torch.Tensor] = None, norm: Optional[bool] = None, eps: float = 1e-6,
                          layout: str = "half") -> dict:
    """Gradients of qk_norm_rope for the gradients g_q, g_k of its outputs; q and
    k are that call's inputs (not needed without norm). Returns "q", "k" (the
    inputs' dtype) and "q_weight", "k_weight" (fp32, None where no weight was
    given)."""
    lib = load_library()
    hg = _heads(g_q, "g_q")
    T, _, D = g_q.shape
    dtype, dev = g_q.dtype, g_q.device
    hgk = None if g_k is None else _heads(g_k, "g_k", _like_k(g_k, g_q), dtype, dev)
    cfg, pos, tab, wq, wk = _rope_call(g_q, g_k, positions, table, q_weight, k_weight, norm, eps, layout)
    hq = hk = hok = gk = ws = gwq = gwk = None
    need = 0
    if cfg.norm:
        hq = _heads(q, "q", g_q.shape, dtype, dev)
        if g_k is not None:
            hk = _heads(k, "k", g_k.shape, dtype, dev)
    gq, hoq = _new(g_q.shape, dtype, dev)
    if g_k is not None:
        gk, hok = _new(g_k.shape, dtype, dev)
    if wq is not None:
        gwq = _vector(D, torch.float32, dev)
    if wk is not None:
        gwk = _vector(D, torch.float32, dev)
    if gwq is not None or gwk is not None:
        need = lib.qk_norm_rope_backward_workspace_size(cfg, T)
        ws = _vector(need, torch.uint8, dev) if need else None
    _check(lib, lib.qk_norm_rope_backward(
        cfg, hq, hk, hg, hgk, pos, tab, wq, wk, T, hoq, hok, _ptr(gwq), _ptr(gwk), _ptr(ws), need,
        _stream(dev)))
    return {"q": gq, "k": gk, "q_weight": gwq, "k_weight": gwk}


# ---------------------------------------------------------------------------
# the caches
# ---------------------------------------------------------------------------

class KVCache:
    """A pool of pages of keys and values in int8 with one fp32 scale for each
    page and head: keys [pages, kv_heads, page, head_dim], values [pages,
    kv_heads, head_dim, page] (a channel's tokens contiguous), scales [pages,
    kv_heads]. page 16, 32, 64 or 128; head_dim 64, 128 or 256.

    Wraps tensors the caller owns; KVCache.empty allocates them. Which pages
    belong to which sequence is the caller's, in the block tables it passes."""

    def __init__(self, keys: torch.Tensor, values: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if keys.dim() != 4 or not keys.is_cuda:
            raise ValueError("keys must be [pages, kv_heads, page, head_dim] on the GPU")
        n, h, p, d = keys.shape
        dev = keys.device
        self._c = _Cache(_address(keys, "keys", None, torch.int8, dev),
                         _address(values, "values", (n, h, d, p), torch.int8, dev),
                         _address(k_scale, "k_scale", (n, h), torch.float32, dev),
                         _address(v_scale, "v_scale", (n, h), torch.float32, dev), n, h, p, d)
        self.keys, self.values, self.k_scale, self.v_scale = keys, values, k_scale, v_scale
        self.device, self.kv_heads, self.page, self.head_dim = dev, h, p, d

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda") -> "KVCache":
        """An unused cache (contents undefined until tokens are appended)."""
        i8 = dict(dtype=torch.int8, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        return cls(torch.empty((n_pages, kv_heads, page, head_dim), **i8),
                   torch.empty((n_pages, kv_heads, head_dim, page), **i8),
                   torch.empty((n_pages, kv_heads), **f32), torch.empty((n_pages, kv_heads), **f32))


class KVCache4:
    """A pool of pages of keys and values in 4-bit floating point (0, 0.5, 1, 1.5, 2, 3, 4, 6
    and their negatives), two entries a byte, the even channel in the low half: keys, values
    uint8 [pages, kv_heads, page, head_dim / 2]. Keys have a power of two for each 32 channels
    of a token, k_exp uint8 [pages, kv_heads, page, head_dim / 32] (its exponent plus 127; 255
    is NaN), values a scale for each token and head, v_scale fp32 [pages, kv_heads, page]. A
    little more than half of KVCache's memory; an append changes no other token's entries. Sizes
    and use as KVCache's."""

    def __init__(self, keys: torch.Tensor, values: torch.Tensor, k_exp: torch.Tensor, v_scale: torch.Tensor):
        if keys.dim() != 4 or not keys.is_cuda:
            raise ValueError("keys must be [pages, kv_heads, page, head_dim / 2] on the GPU")
        n, h, p, d = keys.shape
        d *= 2
        dev = keys.device
        self._c = _Cache4(_address(keys, "keys", None, torch.uint8, dev),
                          _address(values, "values", keys.shape, torch.uint8, dev),
                          _address(k_exp, "k_exp", (n, h, p, d // 32), torch.uint8, dev),
                          _address(v_scale, "v_scale", (n, h, p), torch.float32, dev), n, h, p, d)
        self.keys, self.values, self.k_exp, self.v_scale = keys, values, k_exp, v_scale
        self.device, self.kv_heads, self.page, self.head_dim = dev, h, p, d

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda") -> "KVCache4":
        """An unused cache (contents undefined until tokens are appended)."""
        u8 = dict(dtype=torch.uint8, device=device)
        rows = (n_pages, kv_heads, page)
        return cls(torch.empty(rows + (head_dim // 2,), **u8), torch.empty(rows + (head_dim // 2,), **u8),
                   torch.empty(rows + (head_dim // 32,), **u8), torch.empty(rows, dtype=torch.float32, device=device))


class CacheBatch:
    """The sequences of a call and its new tokens. Sequence b holds kv_lens[b]
    tokens (the new ones included) in the pages block_table[b]; tokens cu[b] ..
    cu[b + 1] of the call are its last. Without cu every sequence has one.

    block_table [B, max_pages], kv_lens [B], cu [B + 1]: int32 on the GPU.
    max_new: at least every sequence's count of new tokens; left out it is one
    without cu, and with cu as many as the call has (a call of few tokens for each
    of many sequences is faster if told so). A sequence's tokens beyond it are not
    stored, and their rows are NaN. max_kv: about the largest kv_lens (it splits
    the work and never changes what is computed). slots: the new tokens' slots, int64 [T],
    as page_plan and cache_slots give them (an append to a 4-bit cache then looks up no pages).
    """

    def __init__(self, block_table: torch.Tensor, kv_lens: torch.Tensor, max_kv: int,
                 cu: Optional[torch.Tensor] = None, max_new: Optional[int] = None,
                 slots: Optional[torch.Tensor] = None):
        if block_table.dim() != 2 or not block_table.is_cuda:
            raise ValueError("block_table must be [B, max_pages] on the GPU")
        B, pages = block_table.shape
        dev = block_table.device
        if max_new is None:
            max_new = 1 if cu is None else _INT32_MAX       # no sequence has more than the call
        self._c = _Batch(_address(block_table, "block_table", None, torch.int32, dev), pages,
                         _address(kv_lens, "kv_lens", (B,), torch.int32, dev),
                         None if cu is None else _address(cu, "cu", (B + 1,), torch.int32, dev),
                         B, pages, _int32(max_new), _int32(max_kv))
        self.block_table, self.kv_lens, self.cu, self.device = block_table, kv_lens, cu, dev
        self.max_kv, self.max_new, self.slots = max_kv, max_new, slots


def _same_device(cache, batch: CacheBatch):
    if cache.device is not batch.device and cache.device != batch.device:
        raise ValueError(f"the cache is on {cache.device}, the batch on {batch.device}")


def kv_cache_append(cache, batch: CacheBatch, k: torch.Tensor, v: torch.Tensor) -> None:
    """Stores the keys and values k, v [T, kv_heads, head_dim] of the batch's
    tokens, in place. KVCache: a page and head whose new tokens exceed its scale gets a
    larger one and its held entries are rounded again; a NaN or an infinity
    makes the scale of its page and head NaN. KVCache4: a token goes to its slot of
    batch.slots, or, without them, of the batch's tables; a NaN or an infinity makes the
    token's 32 channels (keys) or head (values) NaN."""
    lib = load_library()
    _same_device(cache, batch)
    dtype, dev = k.dtype, cache.device
    if dtype not in _DTYPES:
        _check_heads(k, "k", None, None, dev)
    T = k.shape[0]
    shape = (T, cache.kv_heads, cache.head_dim)
    hk = _heads(k, "k", shape, dtype, dev)
    hv = _heads(v, "v", shape, dtype, dev)
    if isinstance(cache, KVCache4):
        slots = None if batch.slots is None else _address(batch.slots, "slots", (T,), torch.int64, dev)
        _run(lib, dev, lib.kv_cache4_append, cache._c, batch._c, slots, hk, hv, _DTYPES[dtype], T)
        return
    _run(lib, dev, lib.kv_cache_append, cache._c, batch._c, hk, hv, _DTYPES[dtype], T)


def kv_cache_read(cache, batch: CacheBatch, total: int, dtype: torch.dtype = torch.bfloat16,
                  k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """The batch's `total` tokens out of the cache: (k, v), each [total,
    kv_heads, head_dim], as the values the entries stand for. Rows of tokens in no
    sequence are left as k and v hold them (undefined where those are not given)."""
    lib = load_library()
    _same_device(cache, batch)
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16 or float32 (got {dtype})")
    dev = cache.device
    shape = (total, cache.kv_heads, cache.head_dim)
    if k is None:
        k, hk = _new(shape, dtype, dev)
    else:
        hk = _heads(k, "k", shape, dtype, dev)
    if v is None:
        v, hv = _new(shape, dtype, dev)
    else:
        hv = _heads(v, "v", shape, dtype, dev)
    read = lib.kv_cache4_read if isinstance(cache, KVCache4) else lib.kv_cache_read
    _run(lib, dev, read, cache._c, batch._c, hk, hv, _DTYPES[dtype], total)
    return k, v


def cache_attention(cache, batch: CacheBatch, q: torch.Tensor, scale: Optional[float] = None,
                    window: int = 0, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                    workspace: Optional[torch.Tensor] = None):
    """Causal attention of the batch's tokens q [T, heads, head_dim] over the
    cache, which holds them already. window > 0: a token sees the last `window`
    keys, its own among them. scale: head_dim^-0.5 by default. heads is a
    multiple of the cache's kv_heads. Returns out [T, heads, head_dim], with
    return_lse also the log of each row's sum, fp32 [T, heads]. A row that sees
    no key gives zeros and -inf; rows of tokens in no sequence are left as out
    holds them (undefined where it is not given). The softmax weights of a bf16 q are kept to 16
    bits, or to 8 in a sequence whose new tokens times heads / kv_heads are more
    than 128; those of an fp32 q to fp32. (KVCache4: q and weights as sums
    of 6-bit pieces, to 2^-17.9 and 2^-13.9 of the largest of 32 channels or keys, weights to
    2^-7.9 where the 8-bit cache's have 8 bits, both to 2^-21.9 for an fp32 q.)"""
    lib = load_library()
    _same_device(cache, batch)
    dev = cache.device
    hq = _heads(q, "q", None, None, dev)
    shape, dtype = q.shape, q.dtype
    T, heads, D = shape
    if D != cache.head_dim:
        raise ValueError(f"q has heads of {D}, the cache of {cache.head_dim}")
    if out is None:
        out, ho = _new(shape, dtype, dev)
    else:
        ho = _heads(out, "out", shape, dtype, dev)
    lse = _empty_strided((T, heads), (heads, 1), dtype=torch.float32, device=dev) if return_lse else None
    dt = _DTYPES[dtype]
    window = _int32(window)
    four = isinstance(cache, KVCache4)
    if workspace is None:
        size = lib.cache4_attention_workspace_size if four else lib.cache_attention_workspace_size
        need = size(cache._c, batch._c, heads, dt, window, T)
        workspace = _vector(need, torch.uint8, dev) if need else None
    else:
        _need_buffer(workspace, "workspace", None, torch.uint8, dev)
        need = workspace.numel()
    attend = lib.cache4_attention if four else lib.cache_attention
    _run(lib, dev, attend, cache._c, batch._c, hq, heads, dt, T, D ** -0.5 if scale is None else scale, window, ho,
         _ptr(lse), _ptr(workspace), need)
    return (out, lse) if return_lse else out
