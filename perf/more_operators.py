"""What a step of the decoder layer needs next to the sparse FFN and the 8-bit cache, as cases
to be timed and compared:

  plan      the pages of a step's tokens, handed out on the GPU: sequences that end or lose
            drafted tokens give theirs back, new tokens get theirs; lengths, offsets,
            positions and the slot of every token
  norm      the residual's addition and the root-mean-square norm in one pass, its output in
            the input's type or in 8 bits with a scale for each row ("fwd"), and the
            gradient ("bwd")
  append    keys and values into a paged 4-bit cache, and the same tokens read back
  attend    attention of one, a few or a chunk of new tokens over that cache

`run` computes them in plain torch operations (fp32, one rounding at the end) or, with `own`
set, by the package's kernels. `exact` computes the same outputs in 64 bits.

The cache holds 4-bit floating point numbers (sign, two bits of exponent, one of mantissa:
0, 0.5, 1, 1.5, 2, 3, 4, 6), two in a byte, the even channel in the low half. Keys and values
are [pages, kv_heads, page, dim / 2] uint8. Keys have a power of two for each 32 channels of a
token (k_exp, uint8 [pages, kv_heads, page, dim / 32], the exponent plus 127), values an fp32
scale for each token and head (v_scale [pages, kv_heads, page]).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_PAIRS = 4096 * 32768 * 32 * 128        # query tokens x keys x heads x dim of the largest listed case
MOST_SCORES = 4096 * 32768 * 32             # its scores
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def plan(name, seqs, new_max, kv_max, page, ends, seed):
    return dict(name=name, op="plan", seqs=seqs, new_max=new_max, kv_max=kv_max, page=page, ends=ends, ragged=seed)


def norm(name, way, tokens, dim, quant, dtype, residual=True):
    return dict(name=name, op="norm", way=way, tokens=tokens, dim=dim, quant=quant, dtype=dtype, residual=residual)


def cached(name, op, seqs, q_max, kv_max, ragged, heads, kv_heads, dim, page, dtype, window=0):
    return dict(name=name, op=op, seqs=seqs, q_max=q_max, kv_max=kv_max, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, dtype=dtype, window=window)


def listed():
    return [
        # the decode step of 32 sequences: a token each, few of which begin a page
        plan("plan decode", 32, 1, 32768, 64, False, 3),
        # continuous batching: 200 sequences of which some end, some take their places with prompts, some decode
        plan("plan prompts", 200, 1500, 8000, 64, True, 5),
        # one decoded token of the 4096-wide layer: latency
        norm("norm one token", "fwd", 1, 4096, "", "bf16"),
        # a 4096-token chunk whose next product takes 8-bit integers
        norm("norm chunk int8", "fwd", 4096, 4096, "int8", "bf16"),
        # a small fp32 model of odd width, 8-bit floating point
        norm("norm odd f32 e4m3", "fwd", 777, 1001, "e4m3", "f32"),
        # the training step's gradient over a chunk
        norm("norm backward chunk", "bwd", 4096, 4096, "", "bf16"),
        # a decode step of 32 sequences of other lengths: one new token each
        cached("append4 batch", "append", 32, 1, 8192, 7, 32, 8, 128, 64, "bf16"),
        # the last chunk of a 32768-token prompt, which starts inside a page
        cached("append4 chunk", "append", 1, 4095, 32768, 0, 32, 8, 128, 64, "bf16"),
        # one sequence's decode step at the full context
        cached("attend4 one at 32768", "attend", 1, 1, 32768, 0, 32, 8, 128, 64, "bf16"),
        # a decode step of 32 sequences, from a few tokens to the full context
        cached("attend4 batch ragged", "attend", 32, 1, 32768, 3, 32, 8, 128, 64, "bf16"),
        # the last chunk of a 32768-token prompt
        cached("attend4 chunk", "attend", 1, 4096, 32768, 0, 32, 8, 128, 64, "bf16"),
        # a few drafted tokens checked at once, each head with its own keys, a sliding window, fp32
        cached("attend4 drafts window f32", "attend", 7, 5, 5000, 11, 8, 8, 64, 16, "f32", 1000),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["plan", "fwd", "bwd", "append", "decode", "drafts", "chunk"])
    if kind == "plan":
        c = plan("", spread(1, 512), 1 if rng.random() < 0.4 else spread(2, 4096), spread(16, 32768),
                 rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.randint(1, 1 << 20))
        # about the tokens that the largest prompts of a step have, and the tables of 200 sequences
        while c["seqs"] * c["new_max"] > 400000:
            c["new_max"] = (c["new_max"] + 1) // 2
        while c["seqs"] * c["kv_max"] > 1 << 22:
            c["kv_max"] = (c["kv_max"] + 1) // 2
    elif kind in ("fwd", "bwd"):
        dim = rng.choice([256, 1024, 4096, 14336, spread(17, 9000)])
        c = norm("", kind, spread(1, 16384), dim, rng.choice(["", "int8", "e4m3"]) if kind == "fwd" else "", dtype,
                 rng.random() < 0.8)
        while c["tokens"] * dim * (1 if dtype == "bf16" else 2) > 4096 * 4096:
            c["tokens"] = (c["tokens"] + 1) // 2
    else:
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 7, 8])
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


def step_lengths(c):
    """Of every sequence before a planned step: tokens held, tokens kept of them, new tokens."""
    r = random.Random(c["ragged"])
    held, keep, new = [], [], []
    for _ in range(c["seqs"]):
        n = max(1, int(math.exp(r.uniform(0, math.log(c["kv_max"] + 1)))))
        what = r.random() if c["ends"] else 0.9
        held.append(n)
        if what < 0.15:         # ended: its place is free
            keep.append(0)
            new.append(0)
        elif what < 0.3:        # ended: its place goes to a prompt
            keep.append(0)
            new.append(r.randint(1, c["new_max"]))
        elif what < 0.5:        # some of its drafted tokens were refused
            keep.append(max(0, n - r.randint(1, 8)))
            new.append(min(c["new_max"], r.randint(1, 8)))
        else:
            keep.append(n)
            new.append(1 if r.random() < 0.7 else r.randint(1, c["new_max"]))
    return held, keep, new


# ---------------------------------------------------------------------------
# 4-bit floating point
# ---------------------------------------------------------------------------

def to_fp4(x):
    """The codes of x (already divided by its scale), to nearest, ties to the even code; two in a byte."""
    a = x.abs()
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = code.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def from_fp4(codes, dtype=torch.float32):
    values = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=dtype, device=codes.device)
    return torch.stack([values[(codes & 15).long()], values[(codes >> 4).long()]], -1).flatten(-2)


def block_exponents(x):
    """For each 32 channels the least power of two by which none exceeds 6, plus 127."""
    m = x.unflatten(-1, (-1, 32)).abs().amax(-1)
    bits = m.view(torch.int32)
    return ((bits >> 23) - 2 + ((bits & 0x7fffff) > 0x400000)).clamp(min=0).to(torch.uint8)


def power(e, dtype=torch.float32):
    return torch.pow(2.0, e.to(torch.float64) - 127).to(dtype).repeat_interleave(32, -1)


def quantise_keys(x):
    e = block_exponents(x)
    return to_fp4(x / power(e)), e


def quantise_values(x):
    s = x.abs().amax(-1) / torch.full((), 6.0, device=x.device)
    return to_fp4(torch.where(s[..., None] > 0, x / s[..., None], x)), s


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    st = {"case": c}
    if c["op"] == "norm":
        dt, T, D = DTYPES[c["dtype"]], c["tokens"], c["dim"]
        # the residual stream has a few channels that are much larger, as trained layers have them
        loud = 1 + 20 * (torch.rand(D, generator=g, device="cuda") < 0.01)
        st.update(weight=(1 + 0.1 * normal(D)).to(dt), eps=1e-6, x=(normal(T, D)).to(dt), residual=None)
        if c["way"] == "bwd":
            st["x"] = (normal(T, D) * loud).to(dt)
            st["g_y"] = (normal(T, D) * 0.1).to(dt)
            st["g_h"] = (normal(T, D) * 0.1).to(dt) if c["residual"] else None
        elif c["residual"]:
            st["residual"] = (normal(T, D) * loud).to(dt)
        return st

    if c["op"] == "plan":
        held, keep, new = step_lengths(c)
        P = c["page"]
        counts = [-(-n // P) for n in held]
        need = sum(max(0, -(-(k + m) // P) - -(-k // P)) for k, m in zip(keep, new))
        width = max(max(counts), max(-(-(k + m) // P) for k, m in zip(keep, new)))
        pages = sum(counts) + need + 100
        st["block_table"] = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        used = torch.arange(width, device="cuda") < i32(counts)[:, None]
        st["block_table"][used] = order[:sum(counts)]
        st["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        st["free"][:pages - sum(counts)] = order[sum(counts):]
        st["n_free"] = i32([pages - sum(counts), 0])
        st["kv_lens"], st["new"] = i32(held), i32(new)
        st["keep"] = i32(keep) if c["ends"] else None
        st["total"] = sum(new)
        return st

    dt = DTYPES[c["dtype"]]
    new, kv = lengths(c)
    B, K, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    counts = [-(-n // P) for n in kv]
    width, pages = max(counts), sum(counts)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([sum(counts[:b]) for b in range(B)], device="cuda")[:, None] + torch.arange(width, device="cuda")
    used = torch.arange(width, device="cuda") < i32(counts)[:, None]
    st["block_table"] = torch.where(used, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    st["lens"] = i32(kv)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu"] = i32(cu)
    st.update(max_new=max(new), max_kv=max(kv), total=cu[-1])
    T = cu[-1]
    # the step's slot map, as its plan leaves it for every layer
    t = torch.arange(T, dtype=torch.int32, device="cuda")
    b = torch.searchsorted(st["cu"], t, right=True) - 1
    pos = (st["lens"][b] - st["cu"][b + 1] + t).long()
    st["slots"] = st["block_table"][b, pos // P].long() * P + pos % P

    # what earlier steps have left in the cache; a few channels of the keys are larger, as learned keys have them
    loud = 1 + 4 * (torch.rand(D, generator=g, device="cuda") < 0.05)
    st["k_codes"], st["k_exp"] = quantise_keys(normal(pages, K, P, D) * loud)
    st["v_codes"], st["v_scale"] = quantise_values(normal(pages, K, P, D))
    if c["op"] == "append":
        st["k"] = (normal(T, K, D) * loud * 1.2).to(dt)
        st["v"] = (normal(T, K, D) * 1.2).to(dt)
    else:
        st["q"] = normal(T, c["heads"], D).to(dt)
        st.update(scale=D ** -0.5, window=c["window"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def plain_plan(st, table, free):
    P, width, pages = st["case"]["page"], table.shape[1], free.shape[0]
    held, new, n_free = st["kv_lens"].long(), st["new"].long(), st["n_free"][:1].long()
    keep = held if st["keep"] is None else torch.minimum(held, st["keep"].long())
    had, kept = -(-held // P), -(-keep // P)
    lens = keep + new
    need = -(-lens // P)
    i = torch.arange(width, device="cuda")
    if st["keep"] is not None:
        # pages beyond what is kept go back, in the order of sequences and of their pages
        back = (i >= kept[:, None]) & (i < had[:, None]) & (table >= 0) & (table < pages)
        at = torch.where(back.flatten(), n_free + back.flatten().cumsum(0) - 1, pages)
        spare = torch.cat([free, free.new_zeros(1)])
        spare[at] = torch.where(back.flatten(), table.flatten(), spare[at])
        free.copy_(spare[:pages])
        n_free = n_free + back.sum()
    # the free pages from the last one down, in the same order
    takes = (i >= kept[:, None]) & (i < need[:, None])
    nth = takes.flatten().cumsum(0) - 1
    page = torch.where(nth < n_free, free[(n_free - 1 - nth).clamp(min=0)], -1)
    table.copy_(torch.where(takes, page.view_as(table), table))
    wanted = takes.sum()
    left = (n_free - wanted).clamp(min=0)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = keep[b] + t - cu[b]
    slots = table[b, pos // P].long()
    slots = torch.where(slots >= 0, slots * P + pos % P, -1)
    return {"kv_lens": lens.int(), "cu": cu.int(), "n_free": torch.cat([left, (wanted - n_free).clamp(min=0)]).int(),
            "positions": pos.int(), "slots": slots, "block_table": table, "free": free}


def plain_norm(st):
    x = st["x"]
    h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    f = h.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + st["eps"])
    n = f * st["weight"].float()
    q = st["case"]["quant"]
    if not q:
        return {"y": (n * r).to(x.dtype), "h": h}
    # the row's factor r divides out of the entries
    s = n.abs().amax(-1, keepdim=True) / n.new_full((), 127.0 if q == "int8" else 448.0)
    e = torch.where(s > 0, n / s, 0.0)
    e = e.round().to(torch.int8) if q == "int8" else e.to(torch.float8_e4m3fn)
    return {"y": e, "scale": (s * r).squeeze(-1), "h": h}


def plain_norm_backward(st):
    x = st["x"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"])
    xh, g = x * r, st["g_y"].float()
    u = g * st["weight"].float()
    gx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    if st["g_h"] is not None:
        gx = gx + st["g_h"].float()
    return {"x": gx.to(st["x"].dtype), "weight": (g * xh).sum(0)}


def plain_append(st):
    c = st["case"]
    page, at = st["slots"] // c["page"], st["slots"] % c["page"]
    st["k_codes"][page, :, at], st["k_exp"][page, :, at] = quantise_keys(st["k"].float())
    st["v_codes"][page, :, at], st["v_scale"][page, :, at] = quantise_values(st["v"].float())
    k = from_fp4(st["k_codes"][page, :, at]) * power(st["k_exp"][page, :, at])
    v = from_fp4(st["v_codes"][page, :, at]) * st["v_scale"][page, :, at][..., None]
    return {"k": k.to(st["k"].dtype), "v": v.to(st["v"].dtype)}


def plain_attend(st):
    c = st["case"]
    B, H, K, D, N = c["seqs"], c["heads"], c["kv_heads"], c["dim"], st["max_new"]
    G = H // K
    table = st["block_table"].long()
    S = table.shape[1] * c["page"]
    k = from_fp4(st["k_codes"][table]) * power(st["k_exp"][table])
    k = k.permute(0, 2, 4, 1, 3).reshape(B, K, D, S)
    v = from_fp4(st["v_codes"][table]) * st["v_scale"][table][..., None]
    v = v.permute(0, 2, 1, 3, 4).reshape(B, K, S, D)
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
    t = torch.searchsorted(cu, torch.arange(st["total"], device="cuda"), right=True) - 1
    at = torch.arange(st["total"], device="cuda") - cu[t]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, H, D)[t, at]
    return {"out": o.to(st["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, N, H)[t, at]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st, c = state, state["case"]
    if c["op"] == "plan":
        # a step that gives pages back changes the table and the free list: they are copied, so
        # that the step can be planned again
        table, free = (st["block_table"], st["free"]) if st["keep"] is None else (st["block_table"].clone(), st["free"].clone())
        if not own:
            return plain_plan(st, table, free)
        import activation_sparse_ffn_amd as sffn
        p = sffn.page_plan(table, st["kv_lens"], st["new"], free, st["n_free"], c["page"], st["total"], keep_lens=st["keep"])
        return {"kv_lens": p.kv_lens, "cu": p.cu, "n_free": p.n_free, "positions": p.positions, "slots": p.slots,
                "block_table": table, "free": free}
    if not own:
        if c["op"] == "norm":
            return plain_norm(st) if c["way"] == "fwd" else plain_norm_backward(st)
        return plain_append(st) if c["op"] == "append" else plain_attend(st)

    import activation_sparse_ffn_amd as sffn
    if c["op"] == "norm":
        if c["way"] == "bwd":
            return sffn.add_rms_norm_backward(st["x"], st["g_y"], st["weight"], g_h=st["g_h"], eps=st["eps"])
        if c["quant"]:
            y, scale, h = sffn.add_rms_norm(st["x"], st["residual"], st["weight"], eps=st["eps"], quant=c["quant"])
            return {"y": y, "scale": scale, "h": h}
        y, h = sffn.add_rms_norm(st["x"], st["residual"], st["weight"], eps=st["eps"])
        return {"y": y, "h": h}
    cache = sffn.KVCache4(st["k_codes"], st["v_codes"], st["k_exp"], st["v_scale"])
    batch = sffn.CacheBatch(st["block_table"], st["lens"], st["max_kv"], st["cu"], st["max_new"], slots=st["slots"])
    if c["op"] == "append":
        sffn.kv_cache_append(cache, batch, st["k"], st["v"])
        k, v = sffn.kv_cache_read(cache, batch, st["total"], st["k"].dtype)
        return {"k": k, "v": v}
    o, lse = sffn.cache_attention(cache, batch, st["q"], scale=st["scale"], window=st["window"], return_lse=True)
    return {"out": o, "lse": lse}


def work(case):
    c = case
    if c["op"] == "plan":
        held, keep, new = step_lengths(c)
        P, B, T = c["page"], c["seqs"], sum(new)
        back = sum(-(-n // P) - -(-k // P) for n, k in zip(held, keep)) if c["ends"] else 0
        taken = sum(-(-(k + m) // P) - -(-k // P) for k, m in zip(keep, new))
        # lengths in and out, offsets, a page's number read and written, of each token its position and slot
        return {"bytes": (4 if c["ends"] else 3) * 4 * B + 4 * B + 8 * (back + taken) + 12 * T, "flops": 4 * B + 4 * T}
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        T, D = c["tokens"], c["dim"]
        n = T * D
        if c["way"] == "bwd":
            return {"bytes": n * e * (4 if c["residual"] else 3) + D * (e + 4), "flops": 12 * n}
        ins, outs = (2, e) if c["residual"] else (1, 0)
        return {"bytes": n * (ins * e + outs + (1 if c["quant"] else e)) + D * e + (4 * T if c["quant"] else 0),
                "flops": 7 * n}
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    new, kv = lengths(c)
    held = D + D // 32 + 4          # bytes of a token and head in the cache
    if c["op"] == "append":
        T = sum(new)
        return {"bytes": T * (K * (4 * D * e + 2 * held) + 8), "flops": 2 * T * K * D * 4}
    seen = pairs = 0
    for m, n in zip(new, kv):
        w = c["window"] or n
        seen += min(n, m - 1 + w)
        pairs += sum(min(n - m + i + 1, w) for i in range(m))
    return {"bytes": K * held * seen + 2 * sum(new) * H * D * e + 4 * sum(new) * H, "flops": 4 * H * D * pairs}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def nearest_level(q):
    """The nearest 4-bit value to each of q, the even code where two are as near."""
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=q.device)
    a = q.abs().clamp(max=6)
    up = torch.bucketize(a, levels).clamp(max=7)
    down = (up - 1).clamp(min=0)
    far, near = levels[up] - a, a - levels[down]
    code = torch.where((far < near) | ((far == near) & (up % 2 == 0)), up, down)
    return torch.copysign(levels[code], q)


def exact_append(st):
    k = st["k"].double().unflatten(-1, (-1, 32))
    most = k.abs().amax(-1, keepdim=True)
    scale = 2.0 ** torch.ceil(torch.log2(most / 6)).clamp(min=-127)
    k = nearest_level(k / scale) * scale
    v = st["v"].double()
    # the scale is kept in fp32, and entries are the quotient's in fp32
    scale = (v.abs().amax(-1, keepdim=True) / 6).float().double()
    v = nearest_level((v / scale).float().double()) * scale
    return {"k": k.flatten(-2), "v": v}


def exact_norm(st):
    leaf = {n: st[n].double().requires_grad_() for n in ("x", "weight")}
    h = leaf["x"]
    if st["residual"] is not None:
        h = (h + st["residual"].double()).to(st["x"].dtype).double()      # the stream is kept in its type
    y = h / (h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + st["eps"]).sqrt() * leaf["weight"]
    c = st["case"]
    if c["way"] == "bwd":
        loss = (y * st["g_y"].double()).sum()
        if st["g_h"] is not None:
            loss = loss + (h * st["g_h"].double()).sum()
        loss.backward()
        return {n: v.grad for n, v in leaf.items()}
    y, h = y.detach(), h.detach()
    if not c["quant"]:
        return {"y": y, "h": h}
    scale = y.abs().amax(-1) / (127 if c["quant"] == "int8" else 448)
    # whole numbers are compared as such; 8-bit floating point with the quotient before its rounding
    return {"y": None if c["quant"] == "int8" else y / scale[:, None], "scale": scale, "h": h}


def exact_attend(st):
    c = st["case"]
    P, G = c["page"], c["heads"] // c["kv_heads"]
    new, kv = lengths(c)
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device="cuda")

    def values(codes):
        both = codes.long()
        out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
        out[..., 0::2], out[..., 1::2] = levels[both % 16], levels[both // 16]
        return out

    outs, lses, t = [], [], 0
    for m, n, row in zip(new, kv, st["block_table"]):
        pages = row[:-(-n // P)].long()
        o = torch.zeros(m, c["heads"], c["dim"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(m, c["heads"], dtype=torch.float64, device="cuda")
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hidden = key > pos
        if c["window"]:
            hidden |= key <= pos - c["window"]
        for h in range(c["kv_heads"]):
            k = values(st["k_codes"][pages, h]).unflatten(-1, (-1, 32))
            k = (k * torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), st["k_exp"][pages, h].long() - 127)[..., None]).flatten(-2)
            k = k.flatten(0, 1)[:n]
            v = (values(st["v_codes"][pages, h]) * st["v_scale"][pages, h].double()[..., None]).flatten(0, 1)[:n]
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
    if case["op"] == "plan":
        return None             # whole numbers
    st = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(st)
    return exact_append(st) if case["op"] == "append" else exact_attend(st)
