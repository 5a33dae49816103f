"""What an append to the 4-bit cache by slots takes of its batch, where no GPU is needed."""
import activation_sparse_ffn_amd as sffn
from tests.test_attention_binding_cpu import FAKE, batch, heads, refused
from tests.test_cache4_binding_cpu import cache

UNSUPPORTED = sffn.SFFN_ERR_UNSUPPORTED


def test_batches_of_an_append_by_slots():
    lib = sffn.load_library()

    def append(b, T=8, k=None):
        return lib.kv_cache4_append(cache(), b, FAKE, k, k, 1, T, None)

    refused(lib, append(batch(n_seqs=-1)), says="n_seqs and max_new")
    refused(lib, append(batch(max_new=-1)), says="n_seqs and max_new")
    refused(lib, append(batch(cu=FAKE + 2)), says="cu must be 4-byte")
    # no sequence has a token that is stored
    assert append(batch(max_new=0)) == 0
    # what is not read may be anything
    for b in (None, batch(block_table=None, kv_lens=None, table_stride=-1, max_pages=-1, max_kv=-5),
              batch(cu=None, max_new=1), batch(n_seqs=0)):
        refused(lib, append(b), says="k is null")
        refused(lib, append(b, T=(1 << 28) + 1, k=heads(st=1024)), UNSUPPORTED, "too large")
