"""What is measured of the operators between the encoder's ids and a model's attention.

  block_tables     pages, slots and positions of new tokens, from request lengths on the GPU
  qk_norm_rope     norms of queries and keys per head with the position rotation, and its backward pass
  tree_attention   attention of new tokens (a tree of drafts, a chain, one token) over a paged cache

Sizes: the ragged requests are the shape of this repository's ragged workload (4,096 requests of 512 to 8,192
bytes, about four bytes a token); heads, pages and context lengths are generic.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step of a small batch: one token each, the launch is all it costs
        dict(name="tables step", op="tables", requests=8, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=4096, page=16, depth=False),
        # the ragged workload's requests admitted at once: 128 to 2,048 tokens each, nothing cached yet
        dict(name="tables prompts", op="tables", requests=4096, new_lo=128, new_hi=2048, ctx_lo=0, ctx_hi=0, page=64, depth=False),
        # a step with drafted trees over long contexts: wide tables, small pages
        dict(name="tables drafts", op="tables", requests=512, new_lo=5, new_hi=31, ctx_lo=1000, ctx_hi=130000, page=16, depth=True),
        # a decode step: eight tokens, keys and values straight into the cache
        dict(name="norm step", op="norm", form="cache", dtype="bf16", tokens=8, hq=32, hk=8, dim=128, rot=128, inter=False, page=16, base=500000.0, far=131072),
        # a prompt batch of the ragged workload's size class
        dict(name="norm prompts", op="norm", form="cache", dtype="bf16", tokens=16384, hq=32, hk=8, dim=128, rot=128, inter=False, page=64, base=500000.0, far=32768),
        # the backward pass of a training batch
        dict(name="norm gradient", op="norm", form="grad", dtype="bf16", tokens=8192, hq=32, hk=8, dim=128, rot=128, inter=False, page=0, base=10000.0, far=8192),
        # an odd count of tokens, narrow heads, interleaved pairs, half of each head rotated
        dict(name="norm gradient odd", op="norm", form="grad", dtype="f16", tokens=777, hq=16, hk=2, dim=64, rot=32, inter=True, page=0, base=10000.0, far=4096),
        # one request, one token: latency
        dict(name="attention one", op="attention", kind="step", dtype="bf16", requests=1, new_lo=1, new_hi=1, ctx_lo=4000, ctx_hi=4000, hq=32, hk=8, dim=128, page=16),
        # a decode step of a large ragged batch
        dict(name="attention batch", op="attention", kind="step", dtype="bf16", requests=128, new_lo=1, new_hi=1, ctx_lo=64, ctx_hi=32768, hq=32, hk=8, dim=128, page=64),
        # drafted trees of a batch verified at once
        dict(name="attention trees", op="attention", kind="tree", dtype="bf16", requests=32, new_lo=16, new_hi=64, ctx_lo=500, ctx_hi=16384, hq=32, hk=8, dim=128, page=64),
        # one long context with a tree of more than 64 drafts, narrow heads
        dict(name="attention long", op="attention", kind="tree", dtype="f16", requests=1, new_lo=100, new_hi=100, ctx_lo=131001, ctx_hi=131001, hq=40, hk=8, dim=64, page=128),
        # prompts in chunks: a chain of new tokens on top of a short context
        dict(name="attention prompts", op="attention", kind="chain", dtype="bf16", requests=4, new_lo=501, new_hi=2048, ctx_lo=0, ctx_hi=1000, hq=32, hk=8, dim=128, page=32),
    ]


HEADS = [(32, 8, 128), (8, 1, 128), (16, 2, 64), (28, 4, 128), (40, 8, 64), (14, 14, 64), (8, 4, 256), (20, 4, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "norm", "attention"])
    if op == "tables":
        n, hi = _log(rng, 1, 4096), _log(rng, 1, 2048)
        ctx = 0 if rng.random() < 0.3 else _log(rng, 1, 130000)
        page = rng.choice([8, 16, 24, 32, 64, 128, 256])
        while n * (ctx + hi) / page > 4e6:  # table entries
            n = max(1, n // 2)
        return dict(op=op, requests=n, new_lo=_log(rng, 1, hi), new_hi=hi, ctx_lo=ctx // rng.randint(1, 50), ctx_hi=ctx, page=page, depth=rng.random() < 0.3)
    hq, hk, dim = rng.choice(HEADS)
    if op == "norm":
        form, inter = rng.choice(["cache", "train", "grad"]), rng.random() < 0.4
        dtype = rng.choice(["bf16", "f16"] if form == "cache" else ["bf16", "f16", "f32"])
        return dict(op=op, form=form, dtype=dtype, tokens=_log(rng, 1, 8192), hq=hq, hk=hk, dim=dim, rot=rng.choice([dim, dim, dim // 2]), inter=inter,
                    page=rng.choice([16, 32, 64, 128]), base=rng.choice([10000.0, 500000.0, 1000000.0]), far=_log(rng, 512, 1000000))
    kind, dtype, page = rng.choice(["step", "tree", "chain"]), rng.choice(["bf16", "f16"]), rng.choice([16, 32, 64, 128, 256])
    n, hi = _log(rng, 1, 128), {"step": 1, "tree": _log(rng, 2, 128), "chain": _log(rng, 1, 2048)}[kind]
    ctx = 0 if rng.random() < 0.1 else _log(rng, 1, 131072)
    while n > 1 and (n * (ctx + hi) * hk * dim > 1.5e9 or n * hi * hq * (ctx + hi) > 4e8):
        n //= 2
    while n * hi * hq * (ctx + hi) > 8e8:
        ctx //= 2
    return dict(op=op, kind=kind, dtype=dtype, requests=n, new_lo=_log(rng, 1, hi), new_hi=hi, ctx_lo=ctx // rng.randint(1, 50), ctx_hi=ctx, hq=hq, hk=hk, dim=dim, page=page)


def _spread(n, lo, hi):
    """n lengths from lo to hi, even over their logarithm (their sum is the case's own; a seed only orders them)."""
    if n == 1 or lo == hi:
        return [hi] * n
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (i / (n - 1)))) - 1 for i in range(n)]


def _lengths(case, rnd=None):
    """(new, ctx) of each request; without a random.Random in one fixed pairing, for work()."""
    new, ctx = _spread(case["requests"], case["new_lo"], case["new_hi"]), _spread(case["requests"], case["ctx_lo"], case["ctx_hi"])
    random.Random(1).shuffle(ctx)  # which new length meets which context is the case's own too
    both = list(zip(new, ctx))
    if rnd is not None:
        rnd.shuffle(both)
    return [b[0] for b in both], [b[1] for b in both]


def _blocks(length, page):
    return -(-length // page)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    return {"tables": _prepare_tables, "norm": _prepare_norm, "attention": _prepare_attention}[case["op"]](case, g, rnd)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def _offsets(new):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int64)).to(DEV)


def _prepare_tables(case, g, rnd):
    n, page = case["requests"], case["page"]
    new, ctx = _lengths(case, rnd)
    old = np.array([_blocks(c, page) for c in ctx])
    need = np.array([_blocks(a + c, page) for a, c in zip(new, ctx)]) - old
    width = int((old + need).max()) + 8
    pages = torch.randperm(int(old.sum() + need.sum()) + 64, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < torch.from_numpy(old).to(DEV)[:, None]
    table[held] = pages[: int(old.sum())]
    total = int(sum(new))
    depth = None
    if case["depth"]:
        depth = torch.randint(0, 8, (total,), generator=g, device=DEV, dtype=torch.int32)
    return dict(case=case, q_off=_offsets(new), ctx=_i32(ctx), free=pages[int(old.sum()):].contiguous(), table=table, total=total, depth=depth)


def _inv_freq(case):
    return torch.tensor([case["base"] ** (-2.0 * j / case["rot"]) for j in range(case["rot"] // 2)], dtype=torch.float32).to(DEV)


def _prepare_norm(case, g, rnd):
    n, hq, hk, dim, t = case["tokens"], case["hq"], case["hk"], case["dim"], DTYPES[case["dtype"]]
    # one projection's output holds the three, as a model's does: heads of a token side by side
    qkv = (torch.randn(n, hq + 2 * hk, dim, generator=g, device=DEV) * 1.7).to(t)
    s = dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], inv_freq=_inv_freq(case))
    s["wq"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(t)
    s["wk"] = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(t)
    s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
    if case["form"] == "grad":
        s["gq"] = torch.randn(n, hq, dim, generator=g, device=DEV).to(t)
        s["gk"] = torch.randn(n, hk, dim, generator=g, device=DEV).to(t)
    if case["form"] == "cache":
        pages = _blocks(n, case["page"]) + 3
        s["k_cache"] = torch.zeros(pages, hk, case["page"], dim, dtype=t, device=DEV)
        s["v_cache"] = torch.zeros(pages, hk, case["page"], dim, dtype=t, device=DEV)
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=DEV)[:n].contiguous()
        s["kept"] = {}
    return s


def _prepare_attention(case, g, rnd):
    n, hq, hk, dim, page, t = case["requests"], case["hq"], case["hk"], case["dim"], case["page"], DTYPES[case["dtype"]]
    new, ctx = _lengths(case, rnd)
    blocks = np.array([_blocks(a + c, page) for a, c in zip(new, ctx)])
    pages = int(blocks.sum()) + 5
    # normalised and rotated queries and keys have entries of order one; values likewise
    kc = torch.randn(pages, hk, page, dim, generator=g, device=DEV, dtype=t)
    vc = torch.randn(pages, hk, page, dim, generator=g, device=DEV, dtype=t)
    table = torch.full((n, int(blocks.max())), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(table.shape[1], device=DEV)[None, :] < torch.from_numpy(blocks).to(DEV)[:, None]
    table[used] = torch.randperm(pages, generator=g, device=DEV)[: int(blocks.sum())].to(torch.int32)
    total, widest = int(sum(new)), max(new)
    q = 1.5 * torch.randn(total, hq, dim, generator=g, device=DEV)
    tree = None
    if case["kind"] == "tree":
        # every node's parent is one of the nodes before it; a row's bits are its ancestors and itself
        words = _blocks(widest, 64)
        bits = np.zeros((n, widest, words * 64), dtype=np.uint8)
        pick = np.random.RandomState(rnd.randrange(1 << 30))
        rows = np.arange(n)
        for i in range(widest):
            if i:
                bits[:, i] = bits[rows, pick.randint(0, i, n)]
            bits[:, i, i] = 1
        packed = np.packbits(bits, axis=2, bitorder="little").view(np.int64)
        live = np.arange(widest)[None, :] < np.array(new)[:, None]
        tree = torch.from_numpy(np.ascontiguousarray(packed[live])).to(DEV)
    return dict(case=case, q=q.to(t), k_cache=kc, v_cache=vc, table=table, q_off=_offsets(new), ctx=_i32(ctx), tree=tree, new=new, widest=widest, kept={})


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "tables":
        return _plain_tables(state, case)
    if case["op"] == "attention":
        return _plain_attention(state, case)
    return _plain_gradient(state, case) if case["form"] == "grad" else _plain_norm(state, case)


def _run_own(s, case):
    import byte_level_bpe_amd as B
    if case["op"] == "tables":
        p = B.block_tables(s["q_off"], s["ctx"], s["free"], s["table"], case["page"], s["total"], depth=s["depth"])
        return {"table": s["table"], "slots": p.slots, "positions": p.positions, "requests": p.requests, "seq_len": p.seq_len, "status": p.status}
    if case["op"] == "attention":
        kept = s["kept"]
        if not kept:  # the handle of the cache, which a program keeps
            kept["cache"] = B.PagedCache(s["k_cache"], s["v_cache"])
        out, lse = B.tree_attention(s["q"], kept["cache"], s["table"], s["q_off"], s["ctx"], tree_mask=s["tree"], return_lse=True)
        return {"out": out, "lse": lse}
    rope = dict(eps=EPS, interleaved=case["inter"])
    if case["form"] == "grad":
        dq, dk, dwq, dwk = B.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], **rope)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if case["form"] == "train":
        q, k = B.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], **rope)
        return {"q": q, "k": k}
    kept = s["kept"]
    if not kept:
        kept["cache"] = B.PagedCache(s["k_cache"], s["v_cache"])
    q, _ = B.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], v=s["v"], cache=kept["cache"], slots=s["slots"], **rope)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_tables(s, case):
    page, table, total = case["page"], s["table"], s["total"]
    n, width = table.shape
    off, ctx, free = s["q_off"], s["ctx"].long(), s["free"]
    new = off[1:] - off[:-1]
    bad = (new < 0) | (off[:-1] < 0) | (off[1:] > total) | (ctx < 0) | (ctx + new > 2**31 - 1)
    new, ctx = new.masked_fill(bad, 0), ctx.clamp(min=0)
    old, end = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    full = ~bad & ((end > width) | (old > width))
    need = torch.where(bad | full | (new == 0), 0, end - old)
    start = torch.cumsum(need, 0) - need
    short = (need > 0) & (start + need > free.numel())
    failed = bad | full | short
    need = need.masked_fill(failed, 0)
    new = new.masked_fill(failed, 0)
    # tables
    col = torch.arange(width, device=table.device)[None, :]
    take = (start[:, None] + col - old[:, None]).clamp(0, max(0, free.numel() - 1))
    fresh = free[take] if free.numel() else torch.full_like(table, -1)
    table.copy_(torch.where(col < old[:, None], table, torch.where(col < (old + need)[:, None], fresh, -1)))
    # tokens
    i = torch.arange(total, device=table.device)
    r = torch.searchsorted(off[1:].contiguous(), i, right=True).clamp(max=n - 1)
    live = (i >= off[r]) & (i - off[r] < new[r])
    p = ctx[r] + (i - off[r]).clamp(min=0)
    held = table[r, (p // page).clamp(max=width - 1)].long()
    slots = torch.where(live & (held >= 0), held * page + p % page, -1)
    positions = torch.where(live, p if s["depth"] is None else ctx[r] + s["depth"], 0).to(torch.int32)
    # status: the first failed request's code and index, pages taken, tokens placed
    codes = torch.where(bad, -1, -5)
    first = torch.argmax(failed.to(torch.int32))
    some = failed.any()
    status = torch.stack([torch.where(some, codes[first], 0), torch.where(some, first, -1), need.sum(), new.sum()])
    return {"table": table, "slots": slots, "positions": positions, "requests": torch.where(live, r, -1).to(torch.int32), "seq_len": (ctx + new).to(torch.int32), "status": status}


def _angles(s):
    # the product in 64 bits: a far position's angle keeps nothing of its fraction in 32
    a = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _halves(y, rot, inter):
    return (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., : rot // 2], y[..., rot // 2 : rot])


def _joined(a, b, rest, inter):
    return torch.cat([torch.stack([a, b], dim=-1).flatten(-2) if inter else torch.cat([a, b], dim=-1), rest], dim=-1)


def _norm_rotate(x, w, cos, sin, rot, inter):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a, b = _halves(y, rot, inter)
    return _joined(a * cos - b * sin, b * cos + a * sin, y[..., rot:], inter)


def _plain_norm(s, case):
    cos, sin = _angles(s)
    q = _norm_rotate(s["q"], s["wq"], cos, sin, case["rot"], case["inter"]).to(s["q"].dtype)
    k = _norm_rotate(s["k"], s["wk"], cos, sin, case["rot"], case["inter"]).to(s["k"].dtype)
    if case["form"] == "train":
        return {"q": q, "k": k}
    at, inside = s["slots"] // case["page"], s["slots"] % case["page"]
    s["k_cache"][at, :, inside] = k
    s["v_cache"][at, :, inside] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _norm_gradient(x, g, w, cos, sin, rot, inter):
    t, x, g, w = x.dtype, x.float(), g.float(), w.float()
    a, b = _halves(g, rot, inter)
    dy = _joined(a * cos + b * sin, b * cos - a * sin, g[..., rot:], inter)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, h = x * rstd, dy * w
    dx = rstd * (h - n * (h * n).mean(-1, keepdim=True))
    return dx.to(t), (dy * n).sum((0, 1))


def _plain_gradient(s, case):
    cos, sin = _angles(s)
    dq, dwq = _norm_gradient(s["q"], s["gq"], s["wq"], cos, sin, case["rot"], case["inter"])
    dk, dwk = _norm_gradient(s["k"], s["gk"], s["wk"], cos, sin, case["rot"], case["inter"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_attention(s, case):
    q, kc, vc, table, off, ctx = s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_off"], s["ctx"].long()
    n, hq, hk, dim, page, widest = case["requests"], case["hq"], case["hk"], case["dim"], case["page"], s["widest"]
    grp, new = hq // hk, off[1:] - off[:-1]
    # queries of every request, padded to the widest: [request, kv head, token * group, dim]
    i = torch.arange(widest, device=q.device)[None, :]
    token = (off[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[token].float().view(n, widest, hk, grp, dim).permute(0, 2, 1, 3, 4).reshape(n, hk, widest * grp, dim)
    # keys and values in the order of the block table
    at = table.long().clamp(min=0)
    keys = kc[at].permute(0, 2, 1, 3, 4).reshape(n, hk, -1, dim).float()
    j = torch.arange(keys.shape[2], device=q.device)
    score = torch.matmul(x, keys.transpose(2, 3).contiguous()).mul_(dim ** -0.5).view(n, hk, widest, grp, -1)
    del keys
    # who sees whom: the context, and of the new tokens its ancestors (a chain: those up to itself)
    d = j[None, :] - ctx[:, None]
    if s["tree"] is None:
        seen = (d[:, None, :] <= i[:, :, None]) & (d < new[:, None])[:, None, :]
    else:
        word = s["tree"][token].gather(2, (d.clamp(0, s["tree"].shape[1] * 64 - 1) // 64)[:, None, :].expand(n, widest, -1))
        bit = (word >> (d.clamp(min=0) % 64)[:, None, :]) & 1
        seen = (d < 0)[:, None, :] | ((bit == 1) & (d < new[:, None])[:, None, :])
        del word, bit
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(top.masked_fill(top == -math.inf, 0)))
    total = p.sum(-1, keepdim=True)
    values = vc[at].permute(0, 2, 1, 3, 4).reshape(n, hk, -1, dim).float()
    out = torch.matmul(p.view(n, hk, widest * grp, -1), values).view(n, hk, widest, grp, dim)
    out = torch.where(total > 0, out / total, 0).permute(0, 2, 1, 3, 4).reshape(n, widest, hq, dim)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(n, widest, hq)
    # back to the tokens' order
    t = torch.arange(q.shape[0], device=q.device)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return {"out": out[r, t - off[r]].to(q.dtype), "lse": lse[r, t - off[r]]}


# ---------------------------------------------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "tables":
        new, ctx = _lengths(case)
        page, n, total = case["page"], case["requests"], sum(new)
        old = [_blocks(c, page) for c in ctx]
        end = [_blocks(a + c, page) for a, c in zip(new, ctx)]
        width = max(end) + 8
        need = sum(end) - sum(old)
        tails = n * width - sum(old)
        # a token's slot may lie in a page that the request held before: one entry read a request
        return {"bytes": 8 * (n + 1) + 4 * n + 4 * need + 4 * n + 4 * tails + total * (16 + (4 if case["depth"] else 0)) + 4 * n + 32, "flops": 10 * total}
    if case["op"] == "norm":
        size = 4 if case["dtype"] == "f32" else 2
        rows, dim = case["tokens"] * (case["hq"] + case["hk"]), case["dim"]
        move = {"train": 2, "cache": 2, "grad": 3}[case["form"]] * rows * dim * size
        if case["form"] == "cache":
            move += 2 * case["tokens"] * case["hk"] * dim * size + 8 * case["tokens"]
        return {"bytes": move + 4 * case["tokens"] + 2 * case["rot"] + 2 * dim * (size if case["form"] != "grad" else size + 4), "flops": rows * dim * (24 if case["form"] == "grad" else 9)}
    new, ctx = _lengths(case)
    hq, hk, dim = case["hq"], case["hk"], case["dim"]
    keys = sum(a + c for a, c in zip(new, ctx))
    pairs = sum(a * c + (a * (a + 1) // 2 if case["kind"] == "chain" else a * a) for a, c in zip(new, ctx))
    total, blocks = sum(new), sum(_blocks(a + c, case["page"]) for a, c in zip(new, ctx))
    return {"bytes": 4 * keys * hk * dim + 4 * total * hq * dim + 4 * total * hq + 4 * blocks + 12 * case["requests"] + 8, "flops": 4 * pairs * hq * dim}


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: equal or wrong
    s = prepare(case, seed)
    return _exact_attention(s, case) if case["op"] == "attention" else _exact_norm(s, case)


def _turn(x, w, turn, rot, inter):
    """The definition: the row over its root mean square, times w, its pairs as complex numbers times exp(i angle)."""
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    head = y[..., :rot]
    pair = head.unflatten(-1, (rot // 2, 2)) if inter else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    head = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
    return torch.cat([head, y[..., rot:]], dim=-1)


def _exact_norm(s, case):
    a = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    turn, rot, inter = torch.polar(torch.ones_like(a), a), case["rot"], case["inter"]
    if case["form"] == "grad":
        got = {}
        for n in "qk":
            x, w = s[n].double().contiguous().requires_grad_(), s["w" + n].double().requires_grad_()
            got["d" + n], got["dw" + n] = torch.autograd.grad(_turn(x, w, turn, rot, inter), (x, w), s["g" + n].double())
        return got
    q, k = (_turn(s[n].double(), s["w" + n].double(), turn, rot, inter) for n in "qk")
    if case["form"] == "train":
        return {"q": q, "k": k}
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for cache, x in ((kc, k), (vc, s["v"].double())):
        flat = cache.transpose(1, 2).reshape(-1, case["hk"], case["dim"])
        flat[s["slots"]] = x
        cache.copy_(flat.view(cache.shape[0], case["page"], case["hk"], case["dim"]).transpose(1, 2))
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_attention(s, case):
    hq, hk, dim, page = case["hq"], case["hk"], case["dim"], case["page"]
    ctx, table = s["ctx"].tolist(), s["table"].cpu()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for r, m in enumerate(s["new"]):
        length = ctx[r] + m
        own_pages = table[r, : _blocks(length, page)].long().to(DEV)
        allowed = torch.ones(m, length, dtype=torch.bool, device=DEV)
        if s["tree"] is None:
            allowed[:, ctx[r]:] = torch.ones(m, m, device=DEV).tril().bool()
        else:
            bits = np.unpackbits(s["tree"][at : at + m].cpu().numpy().view(np.uint8), axis=1, bitorder="little")[:, :m]
            allowed[:, ctx[r]:] = torch.from_numpy(bits.astype(bool)).to(DEV)
        for h in range(hk):
            keys, values = (c[own_pages, h].reshape(-1, dim)[:length].double() for c in (s["k_cache"], s["v_cache"]))
            for e in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = (s["q"][at : at + m, e].double() @ keys.T) / math.sqrt(dim)
                score[~allowed] = -math.inf
                total = torch.logsumexp(score, dim=-1)
                some = total > -math.inf
                lse[at : at + m, e] = total
                out[at : at + m, e] = torch.where(some[:, None], torch.exp(score - total.masked_fill(~some, 0)[:, None]) @ values, 0)
        at += m
    return {"out": out, "lse": lse}
