"""Page bookkeeping where no GPU is needed: refusals of the C entry points and of the
binding."""
import pytest
import torch

import activation_sparse_ffn_amd as sffn
from activation_sparse_ffn_amd import paging as pg
from tests.test_attention_binding_cpu import batch

FAKE = 0x10000      # aligned addresses, never dereferenced: every call here is refused first


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


def pool(**kw):
    base = dict(block_table=FAKE, table_stride=5, free_pages=FAKE, n_pages=10, n_seqs=2, max_pages=5, page=64)
    base.update(kw)
    return pg._Pool(**base)


def refused(lib, status, want=sffn.SFFN_ERR_INVALID_ARG, says=""):
    assert status == want, (status, lib.sparse_ffn_last_error())
    assert says.encode() in lib.sparse_ffn_last_error(), lib.sparse_ffn_last_error()


def plan(lib, p=None, T=4, lens=FAKE, keep=FAKE, new=FAKE + 4, n=FAKE, lens_out=FAKE + 64, n_out=FAKE, cu=FAKE, pos=FAKE,
         slots=FAKE):
    return lib.page_plan(p or pool(), lens, keep, new, n, T, lens_out, n_out, cu, pos, slots, None)


@pytest.mark.parametrize("bad,says,want", [
    (dict(page=48), "page must", 2), (dict(page=256), "page must", 2), (dict(n_pages=0), "n_pages", 1),
    (dict(n_pages=1 << 31), "n_pages", 1), (dict(n_seqs=-1), "n_seqs", 1), (dict(n_seqs=(1 << 24) + 1), "n_seqs", 1),
    (dict(max_pages=0), "max_pages", 1), (dict(max_pages=1 << 25, table_stride=1 << 25), "too many", 2),
    (dict(table_stride=4), "table_stride", 1), (dict(table_stride=-1), "table_stride", 1),
    (dict(block_table=None), "block_table", 1), (dict(block_table=FAKE + 2), "block_table", 1),
    (dict(free_pages=None), "free_pages", 1),
])
def test_pools(lib, bad, says, want):
    refused(lib, plan(lib, pool(**bad)), want, says)


def test_plan_arguments(lib):
    refused(lib, lib.page_plan(None, *[FAKE] * 4, 1, *[FAKE] * 5, None), says="pool")
    refused(lib, plan(lib, T=-1), says="T must")
    refused(lib, plan(lib, T=(1 << 28) + 1), sffn.SFFN_ERR_UNSUPPORTED, says="too large")
    for name, says in (("lens", "kv_lens"), ("new", "new_lens"), ("n", "n_free"), ("lens_out", "kv_lens_out"),
                       ("n_out", "n_free_out"), ("cu", "cu"), ("pos", "positions"), ("slots", "slots")):
        refused(lib, plan(lib, **{name: None}), says=says)
        refused(lib, plan(lib, **{name: FAKE + 2}), says=says)
    refused(lib, plan(lib, slots=FAKE + 4), says="slots")
    refused(lib, plan(lib, keep=FAKE + 1), says="keep_lens")
    refused(lib, plan(lib, lens_out=FAKE + 4), says="kv_lens_out may be")
    refused(lib, plan(lib, keep=FAKE + 64), says="kv_lens_out may be")


def test_slot_arguments(lib):
    def slots(b=None, n_pages=10, page=64, T=4, pos=FAKE, out=FAKE):
        return lib.cache_slots(b or batch(), n_pages, page, T, pos, out, None)

    refused(lib, lib.cache_slots(None, 10, 64, 4, FAKE, FAKE, None), says="batch")
    refused(lib, slots(page=0), sffn.SFFN_ERR_UNSUPPORTED, says="page must")
    refused(lib, slots(n_pages=-1), says="n_pages")
    refused(lib, slots(batch(max_new=-1)), says="max_new")
    refused(lib, slots(batch(max_pages=0)), says="max_pages")
    refused(lib, slots(batch(cu=None)), says="without cu")
    refused(lib, slots(batch(kv_lens=None)), says="kv_lens")
    refused(lib, slots(batch(cu=FAKE + 1)), says="cu")
    refused(lib, slots(pos=None), says="positions")
    refused(lib, slots(out=FAKE + 4), says="slots")
    refused(lib, slots(T=-2), says="T must")
    assert slots(T=0) == sffn.SFFN_OK


def test_binding_refuses_what_it_cannot_pass_on():
    t = torch.zeros(2, 3, dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        sffn.page_plan(t, v, v, v, v, 64, 2)
