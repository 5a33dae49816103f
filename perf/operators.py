"""The attention-side operators of a decoder layer that stand next to the sparse
FFN, as cases to be timed and compared:

  rope      norms of q and k for each head with the position rotation in the
            same pass, forward ("fwd") and backward ("bwd")
  append    new keys and values into a paged 8-bit cache with one scale for each
            page (block of tokens) and head, and the touched tokens read back
  attend    attention of one, a few or a chunk of new tokens over that cache

`run` computes them in plain torch operations (fp32, one rounding at the end)
or, with `own` set, by the package's kernels. `exact` computes the same outputs
in 64 bits.

The cache: keys [pages, kv_heads, page, dim] int8, values [pages, kv_heads, dim,
page] int8 (tokens contiguous), scales [pages, kv_heads] fp32 for each. A
sequence's pages are named by its row of the block table. The batch's new tokens
are the last ones of every sequence: sequence b holds lens[b] tokens, of which
tokens cu[b] .. cu[b + 1] of the call are the last.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_PAIRS = 4096 * 32768 * 32 * 128        # query tokens x keys x heads x dim of the largest listed case
MOST_SCORES = 4096 * 32768 * 32             # its scores


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def rope(name, way, tokens, heads, kv_heads, dim, rot, layout, norm, dtype, packed=False, max_pos=32768):
    return dict(name=name, op="rope", way=way, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot,
                layout=layout, norm=norm, dtype=dtype, packed=packed, max_pos=max_pos)


def cached(name, op, seqs, q_max, kv_max, ragged, heads, kv_heads, dim, page, dtype, window=0):
    return dict(name=name, op=op, seqs=seqs, q_max=q_max, kv_max=kv_max, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, window=window)


def listed():
    return [
        # one decoded token of the 4096-wide layer (32 heads of 128, 8 of them for keys): latency
        rope("rope one token", "fwd", 1, 32, 8, 128, 128, "half", True, "bf16"),
        # a 4096-token chunk of a 32768-token sequence, q and k views of one packed projection
        rope("rope chunk", "fwd", 4096, 32, 8, 128, 128, "half", True, "bf16", packed=True),
        # an fp32 model that rotates a part of each head, interleaved pairs, no norm, an odd count of tokens
        rope("rope part f32", "fwd", 777, 12, 4, 96, 32, "interleaved", False, "f32"),
        # the training step's gradient over a chunk
        rope("rope backward chunk", "bwd", 4096, 32, 8, 128, 128, "half", True, "bf16"),
        # a small fp32 model's gradient, part of the head, interleaved, odd count of tokens
        rope("rope backward f32", "bwd", 1001, 8, 2, 64, 48, "interleaved", True, "f32"),
        # a decode step of 32 sequences of other lengths: one new token each
        cached("append batch", "append", 32, 1, 8192, 7, 32, 8, 128, 64, "bf16"),
        # the last chunk of a 32768-token prompt, which starts inside a page
        cached("append chunk", "append", 1, 4095, 32768, 0, 32, 8, 128, 64, "bf16"),
        # one sequence's decode step at the full context
        cached("attend one at 32768", "attend", 1, 1, 32768, 0, 32, 8, 128, 64, "bf16"),
        # a decode step of 32 sequences, from a few tokens to the full context
        cached("attend batch ragged", "attend", 32, 1, 32768, 3, 32, 8, 128, 64, "bf16"),
        # the last chunk of a 32768-token prompt
        cached("attend chunk", "attend", 1, 4096, 32768, 0, 32, 8, 128, 64, "bf16"),
        # a few drafted tokens checked at once, each head with its own keys, a sliding window, fp32
        cached("attend drafts window f32", "attend", 7, 5, 5000, 11, 8, 8, 64, 16, "f32", 1000),
        # a mixed step: single tokens and chunks of prompts together, 7 query heads to one of keys
        cached("attend mixed", "attend", 6, 1500, 6001, 5, 28, 4, 128, 32, "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["fwd", "bwd", "append", "decode", "drafts", "chunk"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if kind in ("fwd", "bwd"):
        dim = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim // 2, 16 * rng.randint(1, dim // 16)])
        c = rope("", kind, spread(1, 4096), kv_heads * group, kv_heads, dim, rot,
                 rng.choice(["half", "interleaved"]), rng.random() < 0.7, dtype, rng.random() < 0.5,
                 rng.choice([4096, 32768]))
        while c["tokens"] * c["heads"] * c["dim"] > 4096 * 32 * 128:
            c["tokens"] = (c["tokens"] + 1) // 2
    else:
        dim, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
        seqs = 1 if rng.random() < 0.3 else spread(2, 32)
        kv_max = spread(1, 32768)
        q_max = 1 if kind == "decode" else rng.randint(2, 16) if kind == "drafts" else spread(1, 4096)
        if kind == "append" and rng.random() < 0.5:
            q_max = 1
        q_max = min(q_max, kv_max)
        window = spread(16, 4096) if kind != "append" and rng.random() < 0.3 else 0
        c = cached("", "append" if kind == "append" else "attend", seqs, q_max, kv_max, rng.randint(0, 1 << 20),
                   kv_heads * group, kv_heads, dim, page, dtype, window)
        # no more than the largest listed case, in work (four times the operations in fp32) and in padded scores
        while (c["op"] == "attend" and (seqs * c["q_max"] * c["kv_max"] * c["heads"] * dim * (4 if dtype == "f32" else 1)
                                        > MOST_PAIRS or seqs * c["q_max"] * c["kv_max"] * c["heads"] > MOST_SCORES)) \
                or (c["op"] == "append" and seqs * c["q_max"] * kv_heads * dim > 4096 * 1024):
            c["q_max"] = (c["q_max"] + 1) // 2
        # the cache at most that of 32 sequences of 32768 tokens of 8 heads of 128
        while seqs * c["kv_max"] * kv_heads * dim > 32 * 32768 * 1024:
            c["kv_max"] = (c["kv_max"] + 1) // 2
        c["q_max"] = min(c["q_max"], c["kv_max"])
    del c["name"]
    return c


def lengths(c):
    """New tokens and cached tokens (new ones included) of every sequence."""
    if not c["ragged"]:
        return [c["q_max"]] * c["seqs"], [c["kv_max"]] * c["seqs"]
    r = random.Random(c["ragged"])
    kv = [c["kv_max"]] + [int(math.exp(r.uniform(0, math.log(c["kv_max"] + 1)))) for _ in range(c["seqs"] - 1)]
    kv = [max(1, min(c["kv_max"], n)) for n in kv]
    new = [min(c["q_max"], kv[0])] + [r.randint(1, min(c["q_max"], n)) for n in kv[1:]]
    return new, kv


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def rotary_table(max_pos, rot, base, factor):
    """cos | sin of position * frequency, fp32 [max_pos, rot]; positions are divided by `factor`."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / factor
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


_tables = {}


def rotary_of(c):
    """The model's table: made once, as a program keeps it."""
    key = (c["max_pos"], c["rot"])
    if key not in _tables:
        _tables[key] = rotary_table(c["max_pos"], c["rot"], 10000.0, 4.0)
    return _tables[key]


def page_scales(x, dims):
    return x.abs().amax(dims) / torch.tensor(127.0, device=x.device)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    st = {"case": c}
    if c["op"] == "rope":
        T, H, K, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        qkv = (normal(T, H + 2 * K, D) * 1.5).to(dt)
        q, k = qkv[:, :H], qkv[:, H:H + K]
        if not c["packed"]:
            q, k = q.contiguous(), k.contiguous()
        st.update(q=q, k=k, table=rotary_of(c), eps=1e-6)
        start = int(torch.randint(0, c["max_pos"] - T + 1, (1,), generator=g, device="cuda"))
        st["positions"] = torch.arange(start, start + T, dtype=torch.int32, device="cuda")
        st["q_weight"] = st["k_weight"] = None
        if c["norm"]:
            st["q_weight"] = (1 + 0.1 * normal(D)).to(dt)
            st["k_weight"] = (1 + 0.1 * normal(D)).to(dt)
        if c["way"] == "bwd":
            st["g_q"], st["g_k"] = normal(T, H, D).to(dt), normal(T, K, D).to(dt)
        return st

    new, kv = lengths(c)
    B, K, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    counts = [-(-n // P) for n in kv]
    width, pages = max(counts), sum(counts)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(counts[:b]) for b in range(B)], device="cuda")[:, None] + torch.arange(width, device="cuda")
    used = torch.arange(width, device="cuda") < torch.tensor(counts, device="cuda")[:, None]
    st["block_table"] = torch.where(used, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    st["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st.update(max_new=max(new), max_kv=max(kv), total=cu[-1])

    # what earlier steps have left in the cache; a few channels of the keys are larger, as learned keys have them
    loud = 1 + 4 * (torch.rand(D, generator=g, device="cuda") < 0.05)
    x = normal(pages, K, P, D) * loud
    st["k_scale"] = page_scales(x, (2, 3))
    st["k_pages"] = (x / st["k_scale"][:, :, None, None]).round().to(torch.int8)
    x = normal(pages, K, D, P)
    st["v_scale"] = page_scales(x, (2, 3))
    st["v_pages"] = (x / st["v_scale"][:, :, None, None]).round().to(torch.int8)
    del x
    T = cu[-1]
    if c["op"] == "append":
        st["k"] = (normal(T, K, D) * loud * 1.2).to(dt)
        st["v"] = (normal(T, K, D) * 1.2).to(dt)
        # the touched tokens: from the start of the first touched page to the end
        back = [n - (n - m) // P * P for m, n in zip(new, kv)]
        cub = [0]
        for n in back:
            cub.append(cub[-1] + n)
        st["cu_back"] = torch.tensor(cub, dtype=torch.int32, device="cuda")
        st.update(max_back=max(back), total_back=cub[-1])
    else:
        st["q"] = normal(T, c["heads"], D).to(dt)
        st.update(scale=D ** -0.5, window=c["window"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def turn(x, cos, sin, rot, layout):
    """The pairs of the first `rot` of x [T, H, D] turned by the angles of cos, sin [T, rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    pairs = torch.stack([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([pairs.flatten(-2), x[..., rot:]], -1)


def plain_rope(st):
    c = st["case"]
    row = st["table"][st["positions"].long()]
    cos, sin = row[:, :c["rot"] // 2], row[:, c["rot"] // 2:]

    def one(x, w):
        n = x.float()
        if w is not None:
            n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
        return turn(n, cos, sin, c["rot"], c["layout"]).to(x.dtype)

    return {"q": one(st["q"], st["q_weight"]), "k": one(st["k"], st["k_weight"])}


def plain_rope_backward(st):
    c = st["case"]
    row = st["table"][st["positions"].long()]
    cos, sin = row[:, :c["rot"] // 2], row[:, c["rot"] // 2:]

    def one(x, w, g):
        gn = turn(g.float(), cos, -sin, c["rot"], c["layout"])
        if w is None:
            return gn.to(x.dtype), None
        r = torch.rsqrt(x.float().square().mean(-1, keepdim=True) + st["eps"])
        xh, u = x.float() * r, gn * w.float()
        gx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
        return gx.to(x.dtype), (gn * xh).sum((0, 1))

    gq, gqw = one(st["q"], st["q_weight"], st["g_q"])
    gk, gkw = one(st["k"], st["k_weight"], st["g_k"])
    out = {"q": gq, "k": gk}
    return out if gqw is None else {**out, "q_weight": gqw, "k_weight": gkw}


def places(st, cu, total):
    """Sequence, page and slot of each token of the call."""
    P = st["case"]["page"]
    t = torch.arange(total, dtype=torch.int32, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = (st["lens"][b] - cu[b + 1] + t).long()
    return b, pos, st["block_table"][b, pos // P].long(), pos % P


def plain_append(st):
    c = st["case"]
    P = c["page"]
    _, _, page, slot = places(st, st["cu"], st["total"])
    K = c["kv_heads"]
    # the touched pages [B, J] (the last one again where a sequence touches fewer) and the tokens they held
    start = (st["lens"] - st["cu"].diff()).long()
    first, last = start // P, (st["lens"].long() - 1) // P
    j = torch.minimum(first[:, None] + torch.arange((st["max_new"] + P - 2) // P + 1, device="cuda"), last[:, None])
    touched = st["block_table"].long().gather(1, j)
    held = (start[:, None] - j * P).clamp(0, P)
    back = places(st, st["cu_back"], st["total_back"])
    outs = []
    for x, pool, scale, values in ((st["k"], st["k_pages"], st["k_scale"], False), (st["v"], st["v_pages"], st["v_scale"], True)):
        most = torch.zeros_like(scale).index_reduce_(0, page, x.float().abs().amax(-1), "amax")
        old = scale[touched]
        s = torch.where((held > 0)[..., None], torch.maximum(old, most[touched] / most.new_full((), 127.0)),
                        most[touched] / most.new_full((), 127.0))
        entries = pool[touched].float()
        ratio = torch.where((held > 0)[..., None] & (s > 0), old / s, 1.0)
        pool[touched] = (entries * ratio[..., None, None]).round().clamp(-127, 127).to(torch.int8)
        scale[touched] = s
        st_ = scale[page][..., None]
        new = torch.where(st_ > 0, x.float() / st_, 0.0).round().clamp(-127, 127).to(torch.int8)
        if values:
            pool[page, :, :, slot] = new
            got = pool[back[2], :, :, back[3]]
        else:
            pool[page, :, slot] = new
            got = pool[back[2], :, back[3]]
        outs.append((got.float() * scale[back[2]][..., None]).to(x.dtype))
    return {"k": outs[0], "v": outs[1], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def plain_attend(st):
    c = st["case"]
    B, H, K, D, N = c["seqs"], c["heads"], c["kv_heads"], c["dim"], st["max_new"]
    G = H // K
    table = st["block_table"].long()
    S = table.shape[1] * c["page"]
    k = st["k_pages"][table].float() * st["k_scale"][table][..., None, None]
    k = k.permute(0, 2, 4, 1, 3).reshape(B, K, D, S)
    v = st["v_pages"][table].float() * st["v_scale"][table][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, K, S, D)
    cu = st["cu"].long()
    i = torch.arange(N, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=st["total"] - 1)
    q = st["q"].float()[rows].view(B, N, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * N, D)
    pos = (st["lens"] - st["cu"].diff()).long()[:, None] + i
    keys = torch.arange(S, device="cuda")
    sees = (keys <= pos[..., None]) & (keys < st["lens"].long()[:, None, None])
    if st["window"]:
        sees &= keys > pos[..., None] - st["window"]
    s = torch.matmul(q, k).mul_(st["scale"]).view(B, K, G, N, S)
    s = s.masked_fill_(~sees[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, K, G * N, S), v).view(B, K, G, N, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    t, _, _, _ = places(st, st["cu"], st["total"])
    at = torch.arange(st["total"], device="cuda") - cu[t]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, H, D)[t, at]
    return {"out": o.to(st["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, N, H)[t, at]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st, c = state, state["case"]
    if not own:
        if c["op"] == "rope":
            return plain_rope(st) if c["way"] == "fwd" else plain_rope_backward(st)
        return plain_append(st) if c["op"] == "append" else plain_attend(st)

    import activation_sparse_ffn_amd as sffn
    if c["op"] == "rope":
        how = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], norm=c["norm"], eps=st["eps"], layout=c["layout"])
        if c["way"] == "fwd":
            q, k = sffn.qk_norm_rope(st["q"], st["k"], st["positions"], st["table"], **how)
            return {"q": q, "k": k}
        got = sffn.qk_norm_rope_backward(st["q"], st["k"], st["g_q"], st["g_k"], st["positions"], st["table"], **how)
        return {n: t for n, t in got.items() if t is not None}
    cache = sffn.KVCache(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
    batch = sffn.CacheBatch(st["block_table"], st["lens"], st["max_kv"], st["cu"], st["max_new"])
    if c["op"] == "append":
        sffn.kv_cache_append(cache, batch, st["k"], st["v"])
        back = sffn.CacheBatch(st["block_table"], st["lens"], st["max_kv"], st["cu_back"], st["max_back"])
        k, v = sffn.kv_cache_read(cache, back, st["total_back"], st["k"].dtype)
        return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    o, lse = sffn.cache_attention(cache, batch, st["q"], scale=st["scale"], window=st["window"], return_lse=True)
    return {"out": o, "lse": lse}


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "rope":
        T = c["tokens"]
        n, angles = T * (H + K) * D, T * (c["rot"] * 4 + 4)
        if c["way"] == "fwd":
            return {"bytes": 2 * n * e + angles, "flops": n * (8 if c["norm"] else 3)}
        return {"bytes": (3 if c["norm"] else 2) * n * e + angles, "flops": n * (14 if c["norm"] else 3)}
    new, kv = lengths(c)
    if c["op"] == "append":
        held = sum((n - m) % c["page"] for m, n in zip(new, kv))
        T = sum(new)
        # new tokens read; touched tokens: those held before read, all written once; and read back once
        return {"bytes": 2 * K * D * (T * e + held + 2 * (T + held) + (T + held) * e), "flops": 2 * K * D * (6 * T + 4 * held)}
    seen = pairs = 0
    for m, n in zip(new, kv):
        w = c["window"] or n
        seen += min(n, m - 1 + w)
        pairs += sum(min(n - m + i + 1, w) for i in range(m))
    return {"bytes": 2 * K * D * seen + 2 * sum(new) * H * D * e + 4 * sum(new) * H, "flops": 4 * H * D * pairs}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def exact_rope(st):
    c = st["case"]
    R, D = c["rot"], c["dim"]
    angle = st["table"].double()[st["positions"].long()]
    # the rotation as a D x D matrix product on each token: y = n M_t^T
    first = torch.arange(R // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (R // 2 if c["layout"] == "half" else 1)

    def forward(x, w):
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + st["eps"]).sqrt() * w
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle[:, :R // 2], angle[:, R // 2:])[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    leaf = {n: st[n].detach().double().requires_grad_() for n in ("q", "k", "q_weight", "k_weight") if st[n] is not None}
    y = {n: forward(leaf[n], leaf.get(n + "_weight")) for n in ("q", "k")}
    if c["way"] == "fwd":
        return {n: v.detach() for n, v in y.items()}
    ((y["q"] * st["g_q"].double()).sum() + (y["k"] * st["g_k"].double()).sum()).backward()
    return {n: v.grad for n, v in leaf.items()}


def exact_append(st):
    c = st["case"]
    P = c["page"]
    new, kv = lengths(c)
    table = st["block_table"].tolist()
    out = {}
    for n in ("k", "v"):
        pool = st[n + "_pages"].double()
        pool = pool if n == "k" else pool.transpose(2, 3)
        pool, scale, x, got, t = pool.clone(), st[n + "_scale"].double().clone(), st[n].double(), [], 0
        for b in range(c["seqs"]):
            at = kv[b] - new[b]
            while at < kv[b]:
                page, slot = table[b][at // P], at % P
                m = min(P - slot, kv[b] - at)
                piece = x[t:t + m].transpose(0, 1)
                s = (piece.abs().amax((1, 2)) / 127).float().double()
                if slot:
                    s = torch.maximum(s, scale[page])
                    pool[page, :, :slot] = torch.round(pool[page, :, :slot] * (scale[page] / s)[:, None, None])
                pool[page, :, slot:slot + m] = torch.round(piece / s[:, None, None]).clamp(-127, 127)
                scale[page] = s
                at, t = at + m, t + m
            row = torch.tensor(table[b], device="cuda")[(kv[b] - new[b]) // P:-(-kv[b] // P)]
            held = (pool[row] * scale[row][:, :, None, None]).transpose(1, 2).flatten(0, 1)
            got.append(held[:kv[b] - (kv[b] - new[b]) // P * P])
        out[n], out[n + "_scale"] = torch.cat(got), scale
    return out


def exact_attend(st):
    c = st["case"]
    P, D, G = c["page"], c["dim"], c["heads"] // c["kv_heads"]
    new, kv = lengths(c)
    outs, lses, t = [], [], 0
    for m, n, row in zip(new, kv, st["block_table"]):
        pages = row[:-(-n // P)].long()
        o = torch.zeros(m, c["heads"], D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(m, c["heads"], dtype=torch.float64, device="cuda")
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hidden = key > pos
        if c["window"]:
            hidden |= key <= pos - c["window"]
        for h in range(c["kv_heads"]):
            k = (st["k_pages"][pages, h].double() * st["k_scale"][pages, h].double()[:, None, None]).flatten(0, 1)[:n]
            v = (st["v_pages"][pages, h].double() * st["v_scale"][pages, h].double()[:, None, None]).transpose(1, 2).flatten(0, 1)[:n]
            for a in range(h * G, (h + 1) * G):
                s = (st["q"][t:t + m, a].double() * st["scale"]) @ k.T.contiguous()
                s[hidden] = -math.inf
                lse[:, a] = torch.logsumexp(s, 1)
                o[:, a] = (s - lse[:, a, None]).exp() @ v
        outs.append(o)
        lses.append(lse)
        t += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(st)
    return exact_append(st) if case["op"] == "append" else exact_attend(st)
