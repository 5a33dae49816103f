"""What the attention-side entry points promise about sizes, asked of the library
without a GPU."""
import pytest

import activation_sparse_ffn_amd as sffn
from tests.test_attention_binding_cpu import batch, cache

MOST = 256 << 20        # bytes of workspace, whatever the call


@pytest.fixture(scope="module")
def lib():
    return sffn.load_library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [8, 32, 128])
@pytest.mark.parametrize("seqs", [1, 32, 256, 1024, 10000])
def test_workspace_is_bounded(lib, seqs, heads, dim, dtype):
    """Decode steps, drafts and chunks of any count of sequences and any max_kv: the
    parts of rows take at most 256 MiB, and none at all where two would not fit."""
    C = cache(head_dim=dim)
    for new in (1, 2, 8, 40, 300):
        for max_kv in (1000, 32768, 131072, 1 << 20, 2 ** 31 - 1):
            for window in (0, 5000):
                for T in {seqs, seqs * new, 4096}:
                    B = batch(n_seqs=seqs, max_pages=512, table_stride=512, max_new=new, max_kv=max_kv)
                    need = lib.cache_attention_workspace_size(C, B, heads, dtype, window, T)
                    assert need <= MOST, (new, max_kv, window, T, need)


def test_workspace_of_ordinary_calls_is_what_it_was(lib):
    """One sequence of 32768 keys and 32 of them, 32 heads of 128: room for a share of
    512 keys each."""
    for seqs in (1, 32):
        B = batch(n_seqs=seqs, max_pages=512, table_stride=512, max_new=1, max_kv=32768)
        assert lib.cache_attention_workspace_size(cache(), B, 32, 1, 0, seqs) == seqs * 32 * (66 * 130 + 1) * 4
