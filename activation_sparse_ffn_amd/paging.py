"""The pages of a paged cache handed out on the GPU: block tables, lengths, positions and
slots of a step's tokens without a copy to the host, so that a whole step of a model, its
bookkeeping included, can be captured into a graph.

    free, n_free = free_pages(n_pages)
    plan = page_plan(block_table, kv_lens, new_lens, free, n_free, page, total)
    batch = CacheBatch(block_table, plan.kv_lens, max_kv, plan.cu, max_new, slots=plan.slots)
    positions, slots = cache_slots(cache, batch, total)      # of a batch whose pages are there already

A thin ctypes binding of include/sparse_ffn_paging.h, asynchronous on torch's current stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import _run, load_library
from .attention import CacheBatch, _address, _Batch, _vector

__all__ = ["PagePlan", "free_pages", "page_plan", "cache_slots"]

_I32, _I64 = torch.int32, torch.int64


class _Pool(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("free_pages", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page", ctypes.c_int32)]


EXPORTED_SYMBOLS = ("page_plan", "cache_slots")


def declare(lib):
    """The signatures of include/sparse_ffn_paging.h."""
    P, I64, I32, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    lib.page_plan.argtypes = [ctypes.POINTER(_Pool), P, P, P, P, I64, P, P, P, P, P, P]
    lib.page_plan.restype = st
    lib.cache_slots.argtypes = [ctypes.POINTER(_Batch), I64, I32, I64, P, P, P]
    lib.cache_slots.restype = st


class PagePlan(NamedTuple):
    """What page_plan gives: kv_lens [B] after the step, offsets cu [B + 1], n_free [2]
    (pages left, pages lacking), positions [total], all int32, and slots [total] int64."""
    kv_lens: torch.Tensor
    cu: torch.Tensor
    n_free: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor


def free_pages(n_pages: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """All pages of an unused cache: the stack (page 0 on top) and n_free [2]."""
    return (torch.arange(n_pages - 1, -1, -1, dtype=_I32, device=device),
            torch.tensor([n_pages, 0], dtype=_I32, device=device))


def page_plan(block_table: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor, free: torch.Tensor,
              n_free: torch.Tensor, page: int, total: int, keep_lens: Optional[torch.Tensor] = None,
              out: Optional[PagePlan] = None) -> PagePlan:
    """The next step of the sequences of block_table [B, max_pages]: sequence b, which holds
    kv_lens[b] tokens, keeps the first keep_lens[b] of them (None: all; 0 ends it) and gets
    new_lens[b] more. Pages behind those kept go back onto the stack `free` [n_pages], of
    which the first n_free[0] count, and the pages of the new tokens come off its top, in the
    order of sequences; block_table and free change in place. An entry is -1 where no page is
    left (n_free[1] of the result counts them) and such a token's slot is -1: it is not
    stored, and attention over it gives NaN.

    All int32 on one GPU. total: the size of the call that the new tokens are for, at least
    their sum; tokens behind the last sequence's have position 0 and slot -1. out: a plan
    whose tensors take the results; its kv_lens and n_free may be the inputs, so that a
    captured step plans on where it left off."""
    lib = load_library()
    dev = block_table.device
    if block_table.dim() != 2 or not block_table.is_cuda:
        raise ValueError("block_table must be [B, max_pages] on the GPU")
    if free.dim() != 1:
        raise ValueError("free must be [n_pages]")
    B, pages = block_table.shape
    pool = _Pool(_address(block_table, "block_table", None, _I32, dev), pages, _address(free, "free", None, _I32, dev),
                 free.shape[0], B, pages, page)
    lens, fresh = _address(kv_lens, "kv_lens", (B,), _I32, dev), _address(new_lens, "new_lens", (B,), _I32, dev)
    keep = None if keep_lens is None else _address(keep_lens, "keep_lens", (B,), _I32, dev)
    left = _address(n_free, "n_free", (2,), _I32, dev)
    if out is None:
        if total < 0:
            raise ValueError(f"total must not be negative (got {total})")
        # one allocation for what is int32: a call is bound by what the host does
        ints = _vector(2 * B + 3 + total, _I32, dev)
        out = PagePlan(*ints.split_with_sizes((B, B + 1, 2, total)), _vector(total, _I64, dev))
        at = ints.data_ptr()
        to = (at, at + 8 * B + 4, at + 4 * B, at + 8 * B + 12, out.slots.data_ptr())
    else:
        to = (_address(out.kv_lens, "out.kv_lens", (B,), _I32, dev), _address(out.n_free, "out.n_free", (2,), _I32, dev),
              _address(out.cu, "out.cu", (B + 1,), _I32, dev), _address(out.positions, "out.positions", (total,), _I32, dev),
              _address(out.slots, "out.slots", (total,), _I64, dev))
    _run(lib, dev, lib.page_plan, pool, lens, keep, fresh, left, total, *to)
    return out


def cache_slots(cache, batch: CacheBatch, total: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """(positions int32, slots int64) [total] of the batch's tokens in a cache (either kind)
    whose pages its tables name. Tokens of no sequence have position 0 and slot -1; those
    that an append would not store have slot -1."""
    lib = load_library()
    dev = batch.device
    if cache.device != dev:
        raise ValueError(f"the cache is on {cache.device}, the batch on {dev}")
    positions, slots = _vector(total, _I32, dev), _vector(total, _I64, dev)
    _run(lib, dev, lib.cache_slots, batch._c, cache._c.n_pages, cache.page, total, positions.data_ptr(), slots.data_ptr())
    return positions, slots
