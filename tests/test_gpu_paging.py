"""Pages of a step handed out on the GPU, and slots of a batch's tokens, against the
reference that takes one page and token after another (oracle/layer_oracle.py). Whole
numbers: everything is equal."""
import random

import pytest
import torch

from oracle import layer_oracle as lo
from tests.conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(B, kv_max, new_max, page, ends, spare, seed, width=None):
    """Block tables of B sequences, their lengths, what they keep and get, and the stack."""
    r = random.Random(seed)
    held = [r.randint(0, kv_max) for _ in range(B)]
    keep = [r.choice([0, h, max(0, h - r.randint(1, 9)), h + 5]) for h in held] if ends else None
    new = [r.choice([0, 1, 1, r.randint(0, new_max)]) for _ in range(B)]
    counts = [-(-h // page) for h in held]
    width = width or max([1] + [-(-(h + m) // page) for h, m in zip(held, new)])
    counts = [min(c, width) for c in counts]
    n = sum(counts) + spare
    order = list(range(n))
    r.shuffle(order)
    table, at = [], 0
    for c in counts:
        table.append(order[at:at + c] + [-1] * (width - c))
        at += c
    free = order[at:] + [-7] * at
    return table, held, keep, new, free, n - at


def check(table, held, keep, new, free, n_free, page, total, n_out=None):
    import activation_sparse_ffn_amd as sffn
    want = lo.plan(table, held, keep, new, free, n_free, page, total)
    t, f = i32(table), i32(free)
    lens, n = i32(held), i32([n_free, 55])
    p = sffn.page_plan(t, lens, i32(new), f, n, page, total, keep_lens=None if keep is None else i32(keep))
    assert t.tolist() == want[0]
    # above what counts the stack may hold anything
    assert f.tolist()[:want[2]] == want[1][:want[2]]
    assert p.n_free.tolist() == [want[2], want[3]] and p.kv_lens.tolist() == want[4] and p.cu.tolist() == want[5]
    assert p.positions.tolist() == want[6] and p.slots.tolist() == want[7]
    assert lens.tolist() == held and n.tolist() == [n_free, 55]
    return t, p, want


@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,kv_max,new_max", [(1, 300, 1), (1, 0, 5000), (7, 1000, 40), (64, 500, 200), (1023, 60, 3),
                                              (1024, 60, 3), (1025, 60, 20), (2500, 40, 4)])
def test_plans(B, kv_max, new_max, page, ends):
    table, held, keep, new, free, n = state(B, kv_max, new_max, page, ends, 400 + new_max * B // page, B + page)
    for total in {sum(new), sum(new) + 77}:
        check(table, held, keep, new, free, n, page, total)


@pytest.mark.parametrize("spare", [0, 3])
def test_too_few_pages(spare):
    for seed in range(4):
        table, held, keep, new, free, n = state(40, 100, 60, 16, seed % 2 == 1, spare, seed)
        check(table, held, keep, new, free, n, 16, sum(new))


def test_tables_that_end_and_entries_that_name_no_page():
    table, held, keep, new, free, n = state(30, 200, 100, 16, True, 100, 5, width=6)
    for row in table[::3]:
        row[0] = random.Random(1).choice([-1, 1 << 30, len(free)])
    check(table, held, keep, new, free, n, 16, sum(new))
    check(table, [-3] + held[1:], [-1] + keep[1:], [-5] + new[1:], free, n, 16, sum(new))


def test_calls_that_are_too_small():
    """Tokens beyond the call are not written; the sequence that leaves it has no slots."""
    for seed in (1, 2):
        table, held, keep, new, free, n = state(20, 100, 900, 32, False, 800, seed)
        for total in (0, 1, sum(new) // 2, sum(new) - 1):
            check(table, held, keep, new, free, n, 32, total)


@pytest.mark.parametrize("kv_max,new_max,B", [(0, 1, 3), (50, 9000, 5), (40, 30, 3000)])
def test_slots_of_a_batch_are_the_plans(B, kv_max, new_max):
    import activation_sparse_ffn_amd as sffn
    table, held, keep, new, free, n = state(B, kv_max, new_max, 64, False, 1000 + 10 * B, 3)
    total = sum(new) + 5
    t, p, want = check(table, held, keep, new, free, n, 64, total)
    cache = sffn.KVCache.empty(len(free), 1, 64, 64)
    batch = sffn.CacheBatch(t, p.kv_lens, 1, p.cu)
    pos, slots = sffn.cache_slots(cache, batch, total)
    assert pos.tolist() == want[6] and slots.tolist() == want[7]
    # fewer tokens of a sequence than it has
    few = sffn.CacheBatch(t, p.kv_lens, 1, p.cu, max_new=4)
    _, slots = sffn.cache_slots(cache, few, total)
    cut = [-1 if t - want[5][b] >= 4 else want[7][t] for b in range(B) for t in range(want[5][b], want[5][b + 1])]
    assert slots.tolist() == cut + [-1] * 5


def test_slots_of_single_tokens_and_of_offsets_that_leave_the_call():
    import activation_sparse_ffn_amd as sffn
    cache = sffn.KVCache.empty(10, 1, 64, 16)
    table = i32([[3, 4], [9, 12], [1, 2], [5, 6]])
    pos, slots = sffn.cache_slots(cache, sffn.CacheBatch(table, i32([17, 17, 0, 40]), 40), 4)
    assert pos.tolist() == [16, 16, -1, 39] and slots.tolist() == [4 * 16, -1, -1, -1]
    batch = sffn.CacheBatch(table, i32([5, 5, 5, 5]), 5, cu=i32([-2, 3, 3, 5, 9]))
    _, slots = sffn.cache_slots(cache, batch, 7)
    assert slots.tolist() == [-1, -1, -1, 16 + 3, 16 + 4, -1, -1]


def test_a_captured_step_plans_on():
    """The plan's own tensors as its next inputs: replays give what steps one by one give."""
    import activation_sparse_ffn_amd as sffn
    B, page = 5, 16
    free, n_free = sffn.free_pages(64)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    lens = i32([0] * B)
    first = sffn.page_plan(table, lens, i32([3, 20, 16, 1, 15]), free, n_free, page, 55)
    ones = i32([1] * B)
    cap_table, cap_free = table.clone(), free.clone()
    keep = i32([100] * B)
    step = sffn.PagePlan(*(x.clone() for x in (first.kv_lens, first.cu, first.n_free)),
                         torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sffn.page_plan(cap_table, step.kv_lens, ones, cap_free, step.n_free, page, B, keep_lens=keep, out=step)
    kv, n = first.kv_lens, first.n_free
    for i in range(20):
        if i == 9:          # two sequences end, their places begin again
            keep.copy_(i32([100, 0, 100, 0, 100]))
        p = sffn.page_plan(table, kv, ones, free, n, page, B, keep_lens=keep)
        kv, n = p.kv_lens, p.n_free
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(p, step):
            assert torch.equal(a, b)
        assert torch.equal(table, cap_table)
        held = [x for row, m in zip(table.tolist(), kv.tolist()) for x in row[:-(-m // page)]]
        rest = free.tolist()[:n[0].item()]
        assert sorted(held + rest) == list(range(64))       # every page is somewhere, once
        keep.fill_(100)


def test_no_sequences():
    import activation_sparse_ffn_amd as sffn
    free, n_free = sffn.free_pages(4)
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    p = sffn.page_plan(table, i32([]), i32([]), free, n_free, 16, 2)
    assert p.cu.tolist() == [0] and p.n_free.tolist() == [4, 0] and p.slots.tolist() == [-1, -1]


@pytest.mark.parametrize("B,new,page,totals", [(255, 2, 16, (511, 512, 513)), (256, 2, 16, (512, 513)), (257, 7, 16, (2047, 2048, 2049)),
                                               (3, 6000, 16, (16383, 16384, 16400, 18000)), (900, 2, 32, (2048, 2049))])
def test_sizes_around_which_the_plan_is_made_otherwise(B, new, page, totals):
    table, held, keep, fresh, free, n = state(B, 50, new, page, True, 3 * B + B * new // page, 11)
    fresh = [new] * B
    table = [row + [-1] * (1 + new // page) for row in table]
    for total in totals:
        check(table, held, keep, fresh, free, n, page, total)
