"""The operators together, as examples/decoder_layer.py uses them: a prompt taken
in chunks gives what the prompt at once gives. Both round a key or value to 8 bits;
where a page's scale grows between chunks its entries are rounded once more, each
time by at most half a step, 1/254 of the page's largest value, so a few roundings
put about 1/254 sqrt(3) ~ 0.7% of noise on each entry of either side. The layer adds
its input to that, so rel-L2 <= 2e-2 holds for the stream that enters the FFN.

The FFN itself is left out of the comparison: it keeps the largest 16 channels of
each 64, and a channel that is nearly tied changes its place for the smallest
difference of its input (0.4% at the input moves the output of a random FFN by 6%),
so no bound on its output follows from the roundings above."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT, gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts(layer, lengths):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    return [torch.randn(n, layer.d, generator=g, device="cuda").bfloat16() for n in lengths]


class NoFFN:
    """The stream that would enter the FFN comes out as it is."""

    def __call__(self, x):
        return torch.zeros_like(x)


@pytest.mark.parametrize("window", [0, 50])
def test_chunks_and_whole_prompts_agree(example, window):
    layer = example.DecoderLayer(d=512, d_i=2048, heads=4, kv_heads=2, head_dim=64, max_pos=1024)
    layer.ffn = NoFFN()
    ps = prompts(layer, [300, 1, 77])
    whole = example.run(layer, ps, 0, 1000, window)
    for chunk in (64, 37):
        pieces = example.run(layer, ps, 0, chunk, window)
        for a, b in zip(whole, pieces):
            assert a.shape == b.shape and torch.isfinite(a.float()).all()
            d = (a.float() - b.float()).norm() / a.float().norm()
            assert d <= 2e-2, d.item()


def test_decode_steps_follow_a_prompt(example):
    layer = example.DecoderLayer(d=512, d_i=2048, heads=4, kv_heads=2, head_dim=128, max_pos=1024)
    ps = prompts(layer, [130, 63])
    assert all(torch.isfinite(o.float()).all() for o in example.run(layer, ps, 5, 64))
    layer.ffn = NoFFN()
    outs = example.run(layer, ps, 5, 64)
    assert [o.shape[0] for o in outs] == [135, 68]
    # the same tokens as one prompt each: the decode steps' inputs were the outputs before
    again = [torch.cat([p, o[p.shape[0] - 1:-1]]) for p, o in zip(ps, outs)]
    for a, b in zip(example.run(layer, again, 0, 1000), outs):
        assert ((a.float() - b.float()).norm() / b.float().norm()) <= 2e-2
