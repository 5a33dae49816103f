"""Norm, page plan, 4-bit cache and attention in a run, as examples/decoder_layer.py uses
them and as a captured step. A 4-bit entry's scale is its own token's, so a key or value is
stored the same whatever came before it, and a prompt in chunks and at once differ by:

  the projections' fp32 sums of 512 products in another order, at most 2^-15 of their size,
  so that one bf16 result in 2^-15 / 2^-8 * 2 = 2^-6 is off by a step of 2^-8; of these one
  in 2^-5 moves to the next 4-bit code, by a quarter of its value at most: 2^-11 of the
  entries by 2^-2, noise of 2^-5.5 / 4 = 0.6%;
  attention's roundings: 2^-7.9 of the weights, 2^-8 of the output, 0.8%;
  the output projection and the sum with the input, 2^-8 each at the same rare places.

Attention's output is at most as large as the input that the layer adds to it (both have
entries of variance 1 where it sees one key, and more keys average it), so rel-L2 <= 2e-2
holds for the stream that enters the FFN."""
import importlib.util
import os

import pytest
import torch

import activation_sparse_ffn_amd as sffn
from tests.conftest import ROOT, gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class NoFFN:
    def __call__(self, x):
        return torch.zeros_like(x)


@pytest.mark.parametrize("window", [0, 50])
def test_chunks_and_whole_prompts_agree_over_4_bits(example, window):
    layer = example.DecoderLayer(d=512, d_i=2048, heads=4, kv_heads=2, head_dim=64, max_pos=1024)
    layer.ffn = NoFFN()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ps = [torch.randn(n, layer.d, generator=g, device="cuda").bfloat16() for n in (300, 1, 77)]
    whole = example.run(layer, ps, 0, 1000, window, bits=4)
    for chunk in (64, 37):
        for a, b in zip(whole, example.run(layer, ps, 0, chunk, window, bits=4)):
            assert a.shape == b.shape and torch.isfinite(a.float()).all()
            d = (a.float() - b.float()).norm() / a.float().norm()
            assert d <= 2e-2, d.item()


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decoder_layer.py", "--seqs", "2", "--prompt", "40", "--tokens", "2", "--bits", "4"])
    example.main()
    assert "4-bit cache" in capsys.readouterr().out


@pytest.mark.parametrize("bits", [4, 8])
def test_a_captured_step_plans_appends_and_attends(bits):
    """Several tokens by one graph, its lengths and free pages fed back in place: every
    replay gives what the same eager steps give, bit for bit."""
    B, H, Hkv, D, page, pages = 3, 8, 2, 64, 16, 6
    d = H * D
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    steps = torch.randn(20, B, d, generator=g, device="cuda").bfloat16()
    new_kv = torch.randn(20, 2, B, Hkv, D, generator=g, device="cuda").bfloat16()
    weight = torch.rand(d, generator=g, device="cuda").bfloat16()

    class State:
        def __init__(self):
            self.cache = (sffn.KVCache4 if bits == 4 else sffn.KVCache).empty(B * pages, Hkv, D, page)
            for t in ((self.cache.keys, self.cache.values)):
                t.zero_()
            self.table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
            self.free, self.n_free = sffn.free_pages(B * pages)
            self.lens = torch.tensor([0, 5, 15], dtype=torch.int32, device="cuda")
            first = sffn.page_plan(self.table, torch.zeros_like(self.lens), self.lens, self.free, self.n_free, page, 20)
            z = torch.zeros(20, Hkv, D, dtype=torch.bfloat16, device="cuda")
            sffn.kv_cache_append(self.cache, sffn.CacheBatch(self.table, first.kv_lens, 15, first.cu, 15), z, z)
            self.n_free = first.n_free.clone()
            self.one = torch.ones(B, dtype=torch.int32, device="cuda")
            self.plan = sffn.PagePlan(self.lens, torch.zeros(B + 1, dtype=torch.int32, device="cuda"), self.n_free,
                                      torch.zeros(B, dtype=torch.int32, device="cuda"),
                                      torch.zeros(B, dtype=torch.int64, device="cuda"))
            self.x, self.kv = torch.zeros_like(steps[0]), torch.zeros_like(new_kv[0])
            self.h = torch.zeros_like(steps[0])

        def step(self):
            sffn.page_plan(self.table, self.lens, self.one, self.free, self.n_free, page, B, out=self.plan)
            batch = sffn.CacheBatch(self.table, self.lens, page * pages, self.plan.cu, 1, slots=self.plan.slots)
            y, _ = sffn.add_rms_norm(self.x, self.h, weight, h_out=self.h)
            sffn.kv_cache_append(self.cache, batch, self.kv[0], self.kv[1])
            return sffn.cache_attention(self.cache, batch, y.view(B, H, D))

    eager, caught = State(), State()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = State()
        warm.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = caught.step()
    for i in range(20):
        for s in (eager, caught):
            s.x.copy_(steps[i])
            s.kv.copy_(new_kv[i])
        want = eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.isfinite(out.float()).all(), i
        assert torch.equal(eager.table, caught.table) and torch.equal(eager.n_free, caught.n_free)
        assert torch.equal(eager.h, caught.h)
    assert eager.lens.tolist() == [20, 25, 35] and eager.n_free.tolist() == [B * pages - 2 - 2 - 3, 0]
