"""Block tables, the norm of queries and keys with their rotation, and tree
attention on the GPU, against plain forms in 64 bits (tests/serving_reference.py)."""
import math
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import serving_reference as ref  # noqa: E402

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def say(*a):
    print("[gpu-case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def same(got, want, what):
    got, want = got.cpu().numpy(), np.asarray(want)
    assert got.shape == want.shape, what
    bad = np.nonzero((got != want).reshape(-1))[0]
    assert bad.size == 0, (what, int(bad[0]), got.reshape(-1)[bad[0]], want.reshape(-1)[bad[0]], bad.size)


def near(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    off = (got - want).abs()
    ok = (off <= bound) | (got == want)
    assert bool(ok.all()), (what, "worst", float((off / bound)[~ok].nan_to_num(math.inf).max()), "of its bound,", int((~ok).sum()), "values")


# ---------------------------------------------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------------------------------------------
def tables_case(new, ctx, page, width=None, free=None, n_tokens=None, depth=False, seed=0, q_off=None, row_pad=0):
    r = np.random.default_rng(seed)
    n = len(new)
    q_off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64) if q_off is None else np.asarray(q_off, np.int64)
    ctx = np.asarray(ctx, np.int32)
    held = np.maximum(-(-np.maximum(ctx.astype(np.int64), 0) // page), 0)
    need = -(-(np.maximum(ctx.astype(np.int64), 0) + np.asarray(new)) // page)
    width = int(max(need.max() if n else 1, 1)) + 2 if width is None else width
    total = int(q_off[-1]) if n_tokens is None else n_tokens
    count = int(held.sum() + need.sum()) + 5
    pages = r.permutation(count).astype(np.int32)
    table = r.integers(0, 1 << 20, (n, width), dtype=np.int32)  # held entries, and leavings past them
    free_list = pages if free is None else pages[:free]
    d = r.integers(0, 9, total).astype(np.int32) if depth else None
    dev = "cuda"
    store = torch.full((n, width + row_pad), 77, dtype=torch.int32, device=dev)
    t = store[:, :width]
    t.copy_(torch.from_numpy(table))
    got = B.block_tables(torch.from_numpy(q_off).to(dev), torch.from_numpy(ctx).to(dev), torch.from_numpy(free_list.copy()).to(dev), t,
                         page, total, depth=None if d is None else torch.from_numpy(d).to(dev))
    want = ref.tables(q_off, ctx, free_list, table, page, total, d)
    same(t, want[0], "table")
    for name, w in zip(("slots", "positions", "requests", "seq_len", "status"), want[1:]):
        same(getattr(got, name), w, name)
    assert row_pad == 0 or bool((store[:, width:] == 77).all())
    return got, want


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 256])
@pytest.mark.parametrize("n", [1, 2, 63, 513])
def test_block_tables(n, page):
    r = np.random.default_rng(n * 1000 + page)
    say("block_tables", n, page)
    tables_case(r.integers(0, 70, n), r.integers(0, 300, n), page, seed=n, depth=bool(n & 1), row_pad=n % 4)


def test_block_tables_edges():
    for new, ctx in (([0], [0]), ([1], [0]), ([0], [33]), ([16], [16]), ([15, 1, 17], [1, 15, 0]), ([0, 0, 5, 0], [0, 16, 0, 7])):
        say("edges", new, ctx)
        tables_case(new, ctx, 16)
    say("padding past the last request, one token short of a vector")
    tables_case([5, 3], [2, 40], 16, n_tokens=31)
    say("wide rows, rows not 16-byte aligned")
    tables_case([3, 9000], [70000, 5], 8, row_pad=3)
    say("no requests")
    got = B.block_tables(torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                         torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 16, 7)
    assert got.slots.tolist() == [-1] * 7 and got.status.tolist() == [0, -1, 0, 0] and got.positions.tolist() == [0] * 7


@pytest.mark.parametrize("n", [4096, 4097, 9001])
def test_block_tables_many_requests(n):
    r = np.random.default_rng(n)
    say("many", n)
    tables_case(r.integers(0, 9, n), r.integers(0, 40, n), 16, seed=n)
    tables_case(r.integers(0, 9, n), r.integers(0, 40, n), 16, seed=n, free=n // 8)


@pytest.mark.parametrize("n", [6, 4500])
def test_block_tables_failures(n):
    """Free lists that end, full rows, bad contexts and broken offsets: the requests they touch fail, the others do not."""
    new, ctx = np.full(n, 20), np.full(n, 10)
    for free in (0, 1, 4, 5, 7):
        say("free", free)
        got, want = tables_case(new, ctx, 16, free=free)
        if free >= n:  # a page each
            assert got.wait() == (n, n * 20)
            continue
        with pytest.raises(B.BBPEError) as e:
            got.wait()
        assert e.value.status == B.E_CAPACITY and e.value.request == want[5][1]
    say("full rows")
    c = ctx.copy()
    c[2], c[4] = 100, 1000
    tables_case(new, c, 16, width=4)
    say("bad contexts")
    c = ctx.copy()
    c[1], c[3] = -5, 2 ** 31 - 5
    got, _ = tables_case(new, c, 16, width=4)
    with pytest.raises(B.BBPEError) as e:
        got.wait()
    assert e.value.status == B.E_INVALID_ARG and e.value.request == 1
    off = np.concatenate([[0], np.cumsum(new)])
    for at, v in ((0, -1), (3, 1), (5, 10 ** 12), (n, n * 20 + 1), (2, -2 ** 62)):
        say("offset", at, v)
        o = off.copy()
        o[at] = v
        tables_case(new, ctx, 16, q_off=o, n_tokens=n * 20)
    got, _ = tables_case(new, ctx, 16)
    assert got.wait() == (n, n * 20)


@pytest.mark.parametrize("n", [400, 3000, 4096])
def test_block_tables_failures_among_many(n):
    """The same over several workgroups that each scan all requests: with pages for all of them, and too few."""
    r = np.random.default_rng(n)
    new, ctx = r.integers(0, 40, n), r.integers(0, 50, n)
    off = np.concatenate([[0], np.cumsum(new)])
    total = int(off[-1])
    for free in (None, n // 2):
        say("many", n, free)
        tables_case(new, ctx, 16, free=free)
        c = ctx.copy()
        c[n // 3], c[n // 2], c[n - 2] = -1, 1000, 5000
        tables_case(new, c, 16, width=7, free=free)
        for at, v in ((1, -1), (n // 2 + 1, 0), (n // 2 + 1, 2 ** 40), (n - 1, total + 1), (n, -2 ** 63)):
            say("offset", at, v)
            o = off.copy()
            o[at] = v
            tables_case(new, c, 16, width=7, free=free, q_off=o, n_tokens=total)


def test_block_tables_graph_stream_and_outputs():
    """Captured into a graph and replayed with other lengths; on another stream; into given outputs."""
    dev = "cuda"
    say("graph")
    n, page, tokens = 5, 16, 64
    off, ctx = torch.zeros(n + 1, dtype=torch.int64, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    free = torch.arange(100, 140, dtype=torch.int32, device=dev)
    table = torch.zeros(n, 8, dtype=torch.int32, device=dev)
    out = B.block_tables(off, ctx, free, table, page, tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.block_tables(off, ctx, free, table, page, tokens, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.block_tables(off, ctx, free, table, page, tokens, out=out)
    r = np.random.default_rng(0)
    for k in range(4):
        new, c = r.integers(0, 12, n), r.integers(0, 60, n).astype(np.int32)
        t0 = r.integers(0, 50, (n, 8), dtype=np.int32)
        o = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        off.copy_(torch.from_numpy(o))
        ctx.copy_(torch.from_numpy(c))
        table.copy_(torch.from_numpy(t0))
        g.replay()
        torch.cuda.synchronize()
        want = ref.tables(o, c, free.cpu(), t0, page, tokens)
        same(table, want[0], "table")
        for name, w in zip(("slots", "positions", "requests", "seq_len", "status"), want[1:]):
            same(getattr(out, name), w, name)
    say("stream")
    table.copy_(torch.from_numpy(t0))
    torch.cuda.synchronize()
    got = B.block_tables(off, ctx, free, table, page, tokens, stream=side)
    side.synchronize()
    same(got.slots, want[1], "slots on a stream")


# ---------------------------------------------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------------------------------------------
def norm_inputs(n, hq, hk, dim, rot, dtype, seed, far=1000, layout="packed"):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(n, hq + 2 * hk, dim, generator=g) * 2
    wide[:, 0] *= 1e-3  # a row that eps matters for
    if n > 1:
        wide[1, -1] = 0  # a row of zeros
        if hk:
            wide[1, hq] = 0
    wide = wide.to(dtype)
    if layout == "odd":  # rows that are not 16-byte aligned, heads before tokens
        store = torch.zeros(hq + 2 * hk, n, dim + 1, dtype=dtype, device="cuda")
        dev = store.transpose(0, 1)[..., 1:]
        dev.copy_(wide)
    else:
        dev = wide.cuda()
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).to(dtype) for _ in range(2)]
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    freq = torch.tensor([10000.0 ** (-2 * j / max(rot, 1)) for j in range(rot // 2)], dtype=torch.float32)
    return wide, dev, w, pos, freq, g


NORM = [(1, 1, 1, 16, 16, BF, False), (5, 4, 2, 64, 64, BF, False), (7, 3, 1, 128, 128, HF, True), (33, 8, 2, 128, 64, F, False),
        (9, 5, 5, 80, 32, HF, True), (4, 70, 2, 96, 96, BF, False), (3, 2, 1, 256, 256, F, True), (17, 4, 1, 256, 128, BF, False),
        (6, 4, 2, 64, 0, F, False), (2, 3, 0, 32, 32, HF, False), (2, 0, 3, 48, 16, F, True), (0, 4, 2, 64, 64, BF, False),
        (65, 40, 8, 64, 64, HF, False)]


@pytest.mark.parametrize("n,hq,hk,dim,rot,dtype,inter", NORM)
@pytest.mark.parametrize("layout", ["packed", "odd"])
def test_norm_rope(n, hq, hk, dim, rot, dtype, inter, layout):
    say("norm", n, hq, hk, dim, rot, dtype, inter, layout)
    wide, dev, w, pos, freq, _ = norm_inputs(n, hq, hk, dim, rot, dtype, 1, layout=layout)
    wd = [x.cuda() for x in w]
    q, k = B.qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hk], wd[0], wd[1], pos.cuda(), freq.cuda(), eps=1e-5, interleaved=inter)
    for got, x, ww in ((q, wide[:, :hq], w[0]), (k, wide[:, hq:hq + hk], w[1])):
        near(got, *ref.norm_rope(x, ww, pos, freq, 1e-5, inter), "norm")
    say("no weights, in place")
    B.qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hk], None, None, pos.cuda(), freq.cuda(), eps=1e-5, interleaved=inter,
                   q_out=dev[:, :hq], k_out=dev[:, hq:hq + hk])
    near(dev[:, :hq], *ref.norm_rope(wide[:, :hq], None, pos, freq, 1e-5, inter), "in place q")
    near(dev[:, hq:hq + hk], *ref.norm_rope(wide[:, hq:hq + hk], None, pos, freq, 1e-5, inter), "in place k")
    assert torch.equal(dev[:, hq + hk:].cpu(), wide[:, hq + hk:])


def test_norm_rope_far_positions():
    """Angles of positions up to 2^31 - 1, and negative ones, keep their fraction."""
    wide, dev, w, pos, freq, _ = norm_inputs(64, 2, 1, 128, 128, F, 2)
    pos = torch.randint(1 << 20, (1 << 31) - 1, (64,), dtype=torch.int32, generator=torch.Generator().manual_seed(3))
    pos[0], pos[1], pos[2] = (1 << 31) - 1, -1, -(1 << 31)
    say("far")
    q, _ = B.qk_norm_rope(dev[:, :2], dev[:, 2:3], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda())
    near(q, *ref.norm_rope(wide[:, :2], w[0], pos, freq, 1e-6, False), "far positions")


@pytest.mark.parametrize("dim,page,order,dtype", [(64, 16, "heads", BF), (128, 64, "tokens", HF), (256, 1, "heads", BF), (80, 24, "joint", HF)])
def test_norm_rope_into_the_cache(dim, page, order, dtype):
    n, hq, hk, pages = 37, 6, 2, 60 if page < 16 else 7
    say("cache", dim, page, order)
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, dim // 32 * 16, dtype, 5)
    if order == "heads":
        kc, vc = (torch.full((pages, hk, page, dim), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    elif order == "tokens":
        kc, vc = (torch.full((pages, page, hk, dim), 9.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2))
    else:
        both = torch.full((pages, 2, hk, page, dim), 9.0, dtype=dtype, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[3], slots[8], slots[9], slots[10] = -1, pages * page, 1 << 62, -(1 << 62)  # none of these is in the cache
    cache = B.PagedCache(kc, vc)
    q, none = B.qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda(),
                             v=dev[:, hq + hk:], cache=cache, slots=slots.cuda())
    assert none is None
    near(q, *ref.norm_rope(wide[:, :hq], w[0], pos, freq, 1e-6, False), "q")
    yk, bound = ref.norm_rope(wide[:, hq:hq + hk], w[1], pos, freq, 1e-6, False)
    wk, wv = torch.full((pages * page, hk, dim), 9.0, dtype=torch.float64), torch.full((pages * page, hk, dim), 9.0, dtype=torch.float64)
    tol = torch.zeros_like(wk)
    live = (slots >= 0) & (slots < pages * page)
    wk[slots[live]], tol[slots[live]], wv[slots[live]] = yk[live], bound[live], wide[live, hq + hk:].double()
    flat = lambda c: c.transpose(1, 2).reshape(pages * page, hk, dim)  # noqa: E731
    near(flat(kc), wk, tol, "cached keys")
    assert torch.equal(flat(vc).double().cpu(), wv)
    k_out = torch.empty(n, hk, dim, dtype=dtype, device="cuda")
    B.qk_norm_rope(dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda(),
                   v=dev[:, hq + hk:], cache=cache, slots=slots.cuda(), k_out=k_out)
    near(k_out, yk, bound, "k_out beside a cache")


@pytest.mark.parametrize("n,hq,hk,dim,rot,dtype,inter", NORM + [(1500, 4, 2, 64, 64, BF, False)])
@pytest.mark.parametrize("layout", ["packed", "odd"])
def test_norm_rope_backward(n, hq, hk, dim, rot, dtype, inter, layout):
    say("backward", n, hq, hk, dim, rot, dtype, inter, layout)
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, rot, dtype, 7, layout=layout)
    gq, gk = torch.randn(n, hq, dim, generator=g).to(dtype), torch.randn(n, hk, dim, generator=g).to(dtype)
    if n and hk and layout == "odd":  # a broadcast gradient
        gk = gk[:1].expand(n, hk, dim)
    args = (dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda())
    gkd = gk[:1].cuda().expand(n, hk, dim) if n and hk and layout == "odd" else gk.cuda()
    dq, dk, dwq, dwk = B.qk_norm_rope_backward(gq.cuda(), gkd, *args, eps=1e-5, interleaved=inter)
    for dx, dw, gg, x, ww in ((dq, dwq, gq, wide[:, :hq], w[0]), (dk, dwk, gk, wide[:, hq:hq + hk], w[1])):
        a, b = ref.norm_rope_grad(gg, x, ww, pos, freq, 1e-5, inter)
        near(dx, *a, "dx")
        near(dw, *b, "dw")
    say("again: the same bits; without weights; in place")
    again = B.qk_norm_rope_backward(gq.cuda(), gkd, *args, eps=1e-5, interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip((dq, dk, dwq, dwk), again))
    gd = gq.cuda()
    dq, dk, nq, nk = B.qk_norm_rope_backward(gd, gkd, args[0], args[1], None, None, *args[4:], eps=1e-5, interleaved=inter, dq=gd)
    assert nq is None and nk is None and dq is gd
    near(dq, *ref.norm_rope_grad(gq, wide[:, :hq], None, pos, freq, 1e-5, inter)[0], "dx in place")


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_backward_against_differences(inter):
    """The gradient along a direction against central differences of the plain forward in 64 bits."""
    n, hq, hk, dim, rot = 3, 2, 1, 64, 32
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, rot, F, 11)
    gq = torch.randn(n, hq, dim, generator=g)
    say("differences")
    dq, _, dwq, _ = B.qk_norm_rope_backward(gq.cuda(), torch.zeros(n, hk, dim, device="cuda"), dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(),
                                            w[1].cuda(), pos.cuda(), freq.cuda(), interleaved=inter)
    x, ww = wide[:, :hq].double(), w[0].double()
    f = lambda a, b: float((ref.norm_rope(a, b, pos, freq, 1e-6, inter)[0] * gq.double()).sum())  # noqa: E731
    for _ in range(4):
        u = torch.randn(x.shape, generator=g, dtype=torch.float64) * x.abs()  # small rows move little
        z = torch.randn(ww.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        for num, ana in (((f(x + h * u, ww) - f(x - h * u, ww)) / (2 * h), float((dq.double().cpu() * u).sum())),
                         ((f(x, ww + h * z) - f(x, ww - h * z)) / (2 * h), float((dwq.double().cpu() * z).sum()))):
            # differences are good to h^2 and 2^-53 / h, the gradient to 2^-24 a term of some 400
            assert abs(num - ana) <= 1e-4 * max(1.0, abs(num)), (num, ana)


def test_norm_rope_graph():
    n, hq, hk, dim = 19, 4, 2, 64
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, dim, BF, 13)
    a = [dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda()]
    gq, gk = torch.randn(n, hq, dim, device="cuda").to(BF), torch.randn(n, hk, dim, device="cuda").to(BF)
    say("norm graph")

    def step():
        return B.qk_norm_rope(*a) + B.qk_norm_rope_backward(gq, gk, *a)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        dev.mul_(1.25)
        gq.add_(0.5)
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want))


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
def tree_masks(new, words, r, self_too=True):
    """Random trees: every node's parent is one before it."""
    out = []
    for m in new:
        bits = np.zeros((m, words * 64), np.uint8)
        for i in range(m):
            if i:
                bits[i] = bits[r.integers(0, i)]
            if i < words * 64 and self_too:
                bits[i, i] = 1
        out.append(np.packbits(bits, axis=1, bitorder="little").view(np.int64).reshape(m, words))
    return torch.from_numpy(np.concatenate(out) if out else np.zeros((0, words), np.int64))


def attn_inputs(new, ctx, hq, hk, dim, page, dtype, seed=0, words=0, order="heads", sharp=1.5, spare=2):
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    blocks = [-(-(a + c) // page) for a, c in zip(new, ctx)]
    pages = sum(blocks) + spare
    shape = {"heads": (pages, hk, page, dim), "tokens": (pages, page, hk, dim)}[order]
    kc, vc = torch.randn(shape, generator=g).to(dtype), torch.randn(shape, generator=g).to(dtype)
    if order == "tokens":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    perm = r.permutation(pages).astype(np.int32)
    table = np.full((len(new), max(blocks) + 1), -1, np.int32)
    at = 0
    for i, b in enumerate(blocks):
        table[i, :b] = perm[at:at + b]
        at += b
    n = sum(new)
    q = (sharp * torch.randn(n, hq, dim, generator=g)).to(dtype)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    mask = tree_masks(new, words, r) if words else None
    return dict(q=q, k=kc, v=vc, table=torch.from_numpy(table), off=torch.from_numpy(off), ctx=torch.tensor(ctx, dtype=torch.int32),
                mask=mask)


def on_gpu(t):
    d = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return d.copy_(t)


def attn_run(s, scale=None, **kw):
    kc, vc = on_gpu(s["k"]), on_gpu(s["v"])
    return B.tree_attention(s["q"].cuda(), B.PagedCache(kc, vc), s["table"].cuda(), s["off"].cuda(), s["ctx"].cuda(),
                            tree_mask=None if s["mask"] is None else s["mask"].cuda(), scale=scale, return_lse=True, **kw)


def attn_check(s, scale=None, **kw):
    out, lse = attn_run(s, scale, **kw)
    o, tol, l, lt = ref.attention(s["q"], s["k"], s["v"], s["table"], s["off"], s["ctx"], s["mask"], scale)
    near(out, o, tol, "out")
    near(lse, l, lt, "lse")
    return out, lse


ATTN = [  # new, ctx, hq, hk, dim, page, dtype, mask words
    ([1], [0], 1, 1, 64, 16, BF, 0),
    ([1], [1], 4, 1, 128, 16, BF, 0),
    ([1, 1, 1], [31, 128, 257], 8, 2, 128, 16, HF, 0),
    ([1, 1], [1000, 3], 14, 2, 64, 32, BF, 0),
    ([1], [2500], 4, 4, 256, 64, BF, 0),
    ([5, 0, 17], [0, 40, 100], 5, 1, 128, 8, BF, 0),
    ([130, 3], [70, 0], 4, 1, 64, 128, HF, 0),
    ([40], [0], 32, 1, 64, 16, BF, 0),
    ([200], [33], 6, 2, 128, 64, BF, 0),
    ([7, 12, 1], [100, 0, 511], 8, 2, 128, 16, BF, 1),
    ([64, 33], [129, 60], 4, 2, 64, 16, HF, 1),
    ([100], [200], 2, 1, 128, 32, BF, 2),
    ([70], [77], 20, 4, 64, 256, HF, 2),
    ([9], [300], 8, 4, 256, 16, HF, 1),
    ([30], [5], 7, 1, 256, 16, BF, 1),
]


@pytest.mark.parametrize("new,ctx,hq,hk,dim,page,dtype,words", ATTN)
def test_tree_attention(new, ctx, hq, hk, dim, page, dtype, words):
    say("attention", new, ctx, hq, hk, dim, page, dtype, words)
    s = attn_inputs(new, ctx, hq, hk, dim, page, dtype, seed=len(new) + hq, words=words)
    out, lse = attn_check(s)
    again, lse2 = attn_run(s)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_tree_attention_layouts_and_scales():
    say("tokens before heads, odd strides of q and out")
    s = attn_inputs([3, 20], [50, 9], 6, 2, 64, 16, BF, words=1, order="tokens")
    attn_check(s)
    n, hq, dim = s["q"].shape
    odd = torch.zeros(hq, n, dim + 3, dtype=BF, device="cuda").transpose(0, 1)[..., 1:1 + dim]
    odd.copy_(s["q"])
    to = torch.zeros(hq, n, dim + 3, dtype=BF, device="cuda").transpose(0, 1)[..., 1:1 + dim]
    cache = B.PagedCache(on_gpu(s["k"]), on_gpu(s["v"]))
    got = B.tree_attention(odd, cache, s["table"].cuda(), s["off"].cuda(), s["ctx"].cuda(), tree_mask=s["mask"].cuda(), out=to)
    want, _ = attn_run(s)
    assert got is to and torch.equal(got, want)
    for scale in (0.0, -0.3, 2.0):
        say("scale", scale)
        attn_check(s, scale)
    say("a table with strided rows")
    wide = torch.full((2, s["table"].shape[1] + 5), -3, dtype=torch.int32, device="cuda")
    wide[:, :s["table"].shape[1]] = s["table"].cuda()
    got = B.tree_attention(s["q"].cuda(), cache, wide[:, :s["table"].shape[1]], s["off"].cuda(), s["ctx"].cuda(), tree_mask=s["mask"].cuda())
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_tree_attention_empty_rows(dim, dtype):
    """Rows whose mask leaves nothing: zeros and -inf; their neighbours are as ever."""
    s = attn_inputs([9, 5], [0, 37], 4, 2, dim, 16, dtype, words=1)
    s["mask"][2] = 0
    s["mask"][0] = 0
    s["mask"][10] = 0  # has a context still
    say("empty rows", dim, dtype)
    out, lse = attn_check(s)
    assert not out[[0, 2]].any() and bool((lse[[0, 2]] == -math.inf).all()) and bool(torch.isfinite(lse[10]).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,words", [(64, 1), (128, 1), (256, 1), (128, 0)])
def test_tree_attention_masked_places_hold_anything(dim, words, dtype):
    """Infinities, NaN and the type's largest values in places that a row does not see leave it alone; a row that
    sees one has what the formula says."""
    s = attn_inputs([12, 30], [45, 0], 4, 2, dim, 32, dtype, seed=3, words=words)
    clean, lse = attn_run(s)
    kc, vc, table, page = s["k"], s["v"], s["table"], 32
    bad = [math.nan, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).min]
    say("leavings past the last key", dim, words, dtype)
    for r, (c, m) in enumerate(((45, 12), (0, 30))):
        for j in range(c + m, -(-(c + m) // page) * page):
            kc[table[r, j // page], :, j % page] = bad[j % 5]
            vc[table[r, j // page], :, j % page] = bad[(j + 1) % 5]
    kc[-1], vc[-1] = math.nan, math.nan  # and in pages nobody holds, if the last is one
    spare = set(range(kc.shape[0])) - set(table[table >= 0].tolist())
    for p in spare:
        kc[p], vc[p] = math.nan, math.inf
    if kc.shape[0] - 1 not in spare:
        fresh = attn_inputs([12, 30], [45, 0], 4, 2, dim, 32, dtype, seed=3, words=words)
        kc[-1], vc[-1] = fresh["k"][-1], fresh["v"][-1]
        r = int((table == kc.shape[0] - 1).nonzero()[0, 0])
    out, l2 = attn_run(s)
    assert torch.equal(out, clean) and torch.equal(lse, l2)
    say("one new token's values")
    for token, what in ((5, math.nan), (7, math.inf), (8, -math.inf)):
        j = 45 + token
        kk, vv = kc.clone(), vc.clone()
        vv[table[0, j // page], 1, j % page, ::3] = what
        s2 = dict(s, k=kk, v=vv)
        out, l2 = attn_run(s2)
        see = ref.visible(45, 12, None if s["mask"] is None else s["mask"][:12].numpy())[:, j]
        for i in range(12):
            rows = out[i, 2:].float().cpu()
            if see[i]:
                want = torch.full_like(rows[:, ::3], what)
                assert torch.equal(rows[:, ::3].nan_to_num(123.0, 1e30, -1e30), want.nan_to_num(123.0, 1e30, -1e30)), (token, what, i)
                keep = torch.ones(dim, dtype=torch.bool)
                keep[::3] = False
                assert torch.equal(rows[:, keep], clean[i, 2:].float().cpu()[:, keep])
            else:
                assert torch.equal(rows, clean[i, 2:].float().cpu()), (token, what, i)
        assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(out[12:], clean[12:]) and torch.equal(lse, l2)
    say("one new token's key")
    kk = kc.clone()
    kk[table[0, 50 // page], 0, 50 % page] = math.nan
    out, l2 = attn_run(dict(s, k=kk))
    see = torch.from_numpy(ref.visible(45, 12, None if s["mask"] is None else s["mask"][:12].numpy())[:, 50])
    assert bool(out[:12][see.cuda()][:, :2].isnan().all())
    assert torch.equal(out[:12][~see.cuda()], clean[:12][~see.cuda()]) and torch.equal(out[12:], clean[12:])


def test_tree_attention_bad_pages_and_lengths():
    """Pages outside the cache hide their keys; contexts past the row, and negative ones, are cut."""
    s = attn_inputs([4, 6, 3], [100, 40, 64], 4, 2, 64, 16, BF, words=1)
    say("bad pages")
    s["table"][0, 1], s["table"][0, 4], s["table"][1, 0], s["table"][2, 2] = -1, s["k"].shape[0], 2 ** 31 - 1, -2 ** 31
    attn_check(s)
    say("no page at all")
    s["table"][2] = -1
    out, lse = attn_check(s)
    assert not out[10:].any()
    say("a context past the row")
    s = attn_inputs([4, 6, 3], [100, 40, 64], 4, 2, 64, 16, BF, words=1)
    s["ctx"][1] = 10 ** 6
    cut = dict(s, ctx=s["ctx"].clone())
    out, _ = attn_run(cut)
    width = s["table"].shape[1]
    s["table"][1] = torch.arange(width, dtype=torch.int32) % s["k"].shape[0]
    out, lse = attn_run(s)
    o, tol, l, lt = ref.attention(s["q"], s["k"], s["v"], s["table"], s["off"], [100, width * 16, 64], s["mask"])
    near(out, o, tol, "cut context")
    s["ctx"][1] = -7
    out, lse = attn_run(s)
    o, tol, l, lt = ref.attention(s["q"], s["k"], s["v"], s["table"], s["off"], [100, 0, 64], s["mask"])
    near(out, o, tol, "negative context")
    say("offsets that name no tokens of this call")
    s["off"] = torch.tensor([0, 4, 2, 99], dtype=torch.int64)
    out = torch.full_like(s["q"], 7).cuda()
    cache = B.PagedCache(s["k"].cuda(), s["v"].cuda())
    B.tree_attention(s["q"].cuda(), cache, s["table"].cuda(), s["off"].cuda(), s["ctx"].cuda(), tree_mask=s["mask"].cuda(), out=out)
    assert bool((out[4:] == 7).all()) and bool((out[:4] != 7).any())


@pytest.mark.parametrize("dim,words", [(64, 0), (64, 1), (128, 0), (128, 1), (256, 0)])
@pytest.mark.parametrize("hq", [1, 7, 16])
def test_tree_attention_short_tables(dim, words, hq):
    """Table rows about as long as the key counts at which row tiles are cut, or a join is needed at all: full to the
    last key, and with tokens past the row's end."""
    for keys in (32, 128, 160, 256, 320, 384, 400, 512):
        for new in ([1, 1], [2, 60], [30, 33]):
            if keys < 2 * max(new):
                continue
            page = 32 if keys % 128 else 128
            s = attn_inputs(new, [keys - m for m in new], hq, 1, dim, page, BF, words=words, seed=keys)
            s["table"] = s["table"][:, :keys // page].contiguous()
            say("short table", dim, words, hq, keys, new)
            attn_check(s)
            s["ctx"] += torch.tensor([5, 300], dtype=torch.int32)  # the last tokens' own keys are past the row
            out, lse = attn_run(s)
            o, tol, l, lt = ref.attention(s["q"], s["k"], s["v"], s["table"], s["off"], s["ctx"], s["mask"])
            near(out, o, tol, "out past the row")
            near(lse, l, lt, "lse past the row")


ROWS = [
    ([2, 1, 2], 4, 2, 0), ([5, 6], 8, 2, 1), ([1] * 39 + [3], 8, 2, 1), ([1] * 80, 2, 1, 0), ([12, 14], 4, 1, 1),
    ([25, 30], 8, 2, 0), ([70, 50], 4, 1, 2),
]


def rows_check(new, hq, hk, words, dim, dtype, wide):
    page = 32
    ctx = [(77, 0, 45, 131)[r % 4] for r in range(len(new))]
    say("rows", new[:3], hq, hk, words, dim, dtype, wide)
    s = attn_inputs(new, ctx, hq, hk, dim, page, dtype, seed=dim + len(new), words=words)
    if wide:
        table = torch.full((len(new), wide // page), -1, dtype=torch.int32)
        table[:, :s["table"].shape[1]] = s["table"]
        s["table"] = table
    clean, lse = attn_check(s)
    kc, vc, table = s["k"].clone(), s["v"].clone(), s["table"]
    bad = [math.nan, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).min]
    for r, (c, m) in enumerate(zip(ctx, new)):
        for j in range(c + m, -(-(c + m) // page) * page):
            kc[table[r, j // page], :, j % page] = bad[j % 5]
            vc[table[r, j // page], :, j % page] = bad[(j + 1) % 5]
    out, l2 = attn_run(dict(s, k=kc, v=vc))
    assert torch.equal(out, clean) and torch.equal(lse, l2)
    n = new[0]
    j = ctx[0] + n - 1  # the first request's last token
    vc[table[0, j // page], hk - 1, j % page, 1] = math.inf
    out, l2 = attn_run(dict(s, k=kc, v=vc))
    see = torch.from_numpy(ref.visible(ctx[0], n, None if s["mask"] is None else s["mask"][:n].numpy())[:, j]).cuda()
    want = clean.clone()
    rows = want[:n, hq - hq // hk:, 1]
    rows[see] = math.inf
    assert torch.equal(out, want) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new, hq, hk, words", ROWS)
def test_tree_attention_few_and_many_rows(new, hq, hk, words, dim, dtype):
    """Requests of 4 to 240 rows each, for the row tiles of every size: right, and blind to what a row does not see."""
    rows_check(new, hq, hk, words, dim, dtype, None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new, hq, hk, words", ROWS)
def test_tree_attention_few_and_many_rows_in_wide_tables(new, hq, hk, words, dim, dtype):
    """The same where table rows could hold many keys."""
    rows_check(new, hq, hk, words, dim, dtype, 5000 // 32 * 32)


def test_tree_attention_many_requests():
    """More requests than one launch takes, of mixed lengths, most of them short."""
    r = np.random.default_rng(5)
    n = 2300
    new, ctx = [int(x) for x in r.integers(0, 3, n)], [int(x) for x in r.integers(0, 40, n)]
    ctx[7], new[8] = 5000, 60
    say("many requests")
    s = attn_inputs(new, ctx, 2, 1, 64, 16, BF, seed=9)
    attn_check(s)


def test_tree_attention_sharp_scores():
    """Weights of very different size: the maximum sits in the last tile, or scores run to +-2,000."""
    s = attn_inputs([2], [900], 4, 2, 128, 16, BF, sharp=40.0)
    say("sharp")
    attn_check(s)
    s["q"][0, 0] = s["k"][s["table"][0, 900 // 16], 0, 900 % 16] * 30
    attn_check(s)


def test_tree_attention_cache_past_32_bits():
    """Pages that begin past 2^32 elements (8.6 GB into the cache)."""
    page, hk, dim = 256, 8, 128
    per = page * hk * dim
    pages = (1 << 32) // per + 4
    say("large cache", pages)
    kc = torch.empty(pages, hk, page, dim, dtype=BF, device="cuda")
    vc = torch.empty(pages, hk, page, dim, dtype=BF, device="cuda")
    s = attn_inputs([3], [600], 8, 8, dim, page, BF, words=1, spare=0)
    top = torch.tensor([pages - 1, 0, pages - 3], dtype=torch.int32)
    for j in range(3):
        kc[int(top[j])], vc[int(top[j])] = s["k"][int(s["table"][0, j])].cuda(), s["v"][int(s["table"][0, j])].cuda()
    table = s["table"].clone()
    table[0, :3] = top
    cache = B.PagedCache(kc, vc)
    got = B.tree_attention(s["q"].cuda(), cache, table.cuda(), s["off"].cuda(), s["ctx"].cuda(), tree_mask=s["mask"].cuda())
    want, _ = attn_run(s)
    assert torch.equal(got, want)
    say("and writing there")
    slot = torch.tensor([(pages - 1) * page + 255], dtype=torch.int64, device="cuda")
    one = torch.randn(1, 3 * hk, dim, device="cuda").to(BF)
    B.qk_norm_rope(one[:, :hk], one[:, hk:2 * hk], None, None, torch.zeros(1, dtype=torch.int32, device="cuda"),
                   torch.ones(dim // 2, device="cuda"), v=one[:, 2 * hk:], cache=cache, slots=slot)
    assert torch.equal(vc[pages - 1, :, 255], one[0, 2 * hk:])


def test_tree_attention_graph_and_streams():
    s = attn_inputs([2, 9, 1], [700, 33, 0], 8, 2, 128, 16, BF, words=1)
    cache = B.PagedCache(on_gpu(s["k"]), on_gpu(s["v"]))
    q, table, off, ctx, mask = (s[n].cuda() for n in ("q", "table", "off", "ctx", "mask"))
    run = lambda **kw: B.tree_attention(q, cache, table, off, ctx, tree_mask=mask, return_lse=True, **kw)  # noqa: E731
    run()
    torch.cuda.synchronize()
    say("attention graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run()
    for k in range(4):
        q.mul_(0.9)
        ctx.copy_(torch.tensor([700 - 100 * k, 33 + k, 0], dtype=torch.int32))
        want = run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
    say("streams")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])


# ---------------------------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------------------------
def test_text_to_attention():
    """Encoded requests on the device through pages, slots, norm and rotation into the cache, then a step with drafted
    trees on top: every row against 64 bits on what the cache holds."""
    from synth import configs
    w = configs.tiny()
    tok = B.load_ranks(w.tokens, w.specials, w.grammar)
    text = w.segments[0][0]
    segs = [(text[a:b], False) for a, b in ((0, 180), (180, 183), (183, 700), (700, 700), (700, 1400))]
    t, seg_off, allow, total = B.to_device_segments(segs)
    ids, id_off, n = tok.encode_device(t, seg_off, allow, total)
    say("chain of operators", n)
    g = torch.Generator(device="cuda").manual_seed(0)
    hq, hk, dim, page, pages, reqs = 8, 2, 64, 16, 80, len(segs)
    emb = torch.randn(tok.info()["max_id"] + 1, (hq + 2 * hk) * dim, generator=g, device="cuda").to(BF)
    freq = torch.tensor([10000.0 ** (-2 * j / dim) for j in range(dim // 2)], device="cuda")
    wq = torch.ones(dim, dtype=BF, device="cuda") * 1.2
    cache = B.PagedCache(*(torch.full((pages, hk, page, dim), math.nan, dtype=BF, device="cuda") for _ in range(2)))
    table = torch.full((reqs, 48), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    ctx = torch.zeros(reqs, dtype=torch.int32, device="cuda")

    def layer(ids, off, plan, mask):
        x = emb[ids.long()].view(-1, hq + 2 * hk, dim)
        q, _ = B.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], wq, wq, plan.positions, freq, v=x[:, hq + hk:], cache=cache, slots=plan.slots)
        out, lse = B.tree_attention(q, cache, table, off, ctx, tree_mask=mask, return_lse=True)
        o, tol, l, lt = ref.attention(q.cpu(), cache.k.cpu(), cache.v.cpu(), table.cpu(), off.cpu(), ctx.cpu(),
                                      None if mask is None else mask.cpu())
        near(out, o, tol, "out")
        near(lse, l, lt, "lse")

    plan = B.block_tables(id_off, ctx, free, table, page, n)
    taken, placed = plan.wait()
    assert placed == n
    layer(ids, id_off, plan, None)
    ctx = plan.seq_len.clone()
    new = [3, 1, 7, 2, 5]
    off = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int64, device="cuda")
    mask = tree_masks(new, 1, np.random.default_rng(0))
    depth = torch.tensor([bin(int(m) & (2 ** 64 - 1)).count("1") - 1 for m in mask[:, 0].tolist()], dtype=torch.int32, device="cuda")
    plan = B.block_tables(off, ctx, free[taken:].contiguous(), table, page, sum(new), depth=depth)
    plan.wait()
    layer(ids[:sum(new)], off, plan, mask.cuda())


def test_example():
    """examples/serving_step.py: an accepted path is the same as a chain (two roundings of the output and of the
    weights apart: values of order one, bfloat16), and gradients arrive."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    off_by, tree, leaves = mod.main()
    # each side: half a step of the output, and half a step of every weight on values below 8
    assert off_by <= 2 * ref.half_step(BF) * (float(tree.float().abs().max()) + 8)
    assert all(bool(torch.isfinite(t.grad).all()) and bool(t.grad.any()) for t in leaves)
