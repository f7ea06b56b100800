"""tree_attention where row tiles, runs and requests of every kind meet: against
64 bits (tests/serving_dense.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import serving_dense as dense  # noqa: E402
from tests.test_gpu_serving import attn_inputs, attn_run, near, on_gpu, say  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(s, scale=None, **kw):
    out, lse = attn_run(s, scale)
    o, tol, l, lt = dense.attention(s["q"], s["k"], s["v"], s["table"], s["off"], s["ctx"], s["mask"], scale, **kw)
    near(out, o, tol, "out")
    near(lse, l, lt, "lse")
    return out, lse


@pytest.mark.parametrize("n,at,value", [
    (4, 2, 1),         # offsets 0 3 1 9 12: requests 1 (3 to 1) and, by its own offsets alone fine, 2 (1 to 9)
    (4, 3, 10 ** 12),  # past the tokens
    (4, 0, -1),        # the first offset: nobody is served
    (70, 20, 2), (70, 70, 1),
    (2500, 700, 5), (2500, 1024, 7), (2500, 1025, 7), (2500, 1900, 0), (2500, 2500, -5),
])
def test_requests_behind_a_broken_offset(n, at, value):
    """As in block_tables: from the first request whose offsets cannot be followed on none has tokens, whatever its own
    offsets are, in this launch of the kernels and the next ones; the ones before are served."""
    r = np.random.default_rng(n)
    new = [3] * 4 if n == 4 else [int(x) for x in r.integers(0, 3, n)]
    ctx = [int(x) for x in r.integers(0, 20, n)]
    say("broken offset", n, at, value)
    s = attn_inputs(new, ctx, 2, 1, 64, 16, BF, seed=n)
    off = s["off"].clone()
    off[at] = value
    o = off.tolist()
    good = next(q for q in range(n + 1) if q == n or o[q] < 0 or o[q + 1] < o[q] or o[q + 1] > sum(new))
    assert good < n
    served = int(s["off"][good])
    out, lse = torch.full_like(s["q"], 7).cuda(), torch.full(s["q"].shape[:2], 7.0, device="cuda")
    B.tree_attention(s["q"].cuda(), B.PagedCache(on_gpu(s["k"]), on_gpu(s["v"])), s["table"].cuda(), off.cuda(), s["ctx"].cuda(), out=out, lse=lse)
    want, tol, want_lse, lse_tol = dense.attention(s["q"][:served], s["k"], s["v"], s["table"][:good], o[:good + 1], s["ctx"][:good])
    near(out[:served], want, tol, "the requests before")
    near(lse[:served], want_lse, lse_tol, "the requests before")
    assert bool((out[served:] == 7).all()) and bool((lse[served:] == 7).all())


@pytest.mark.parametrize("tokens,hq", [(1, 1), (20, 1), (40, 2), (70, 2), (300, 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("below", [10, 14.5])
def test_small_weights_in_float16(dim, tokens, hq, below):
    """A first key that takes nearly all of the weight and has no values, in front of keys up to 17.45 below: their
    weights, down to 2^-25 of the first's, are what the output is made of.  They are held to 2^-32 of it."""
    say("small weights", dim, tokens, hq, below)
    ctx = 290 if tokens < 300 else 20
    s = attn_inputs([tokens], [ctx], hq, 1, dim, 16, HF, seed=dim + tokens)
    g = torch.Generator().manual_seed(1)
    s["q"].zero_()[..., 0] = 1
    s["k"].zero_()[..., 0] = -below - (17.45 - below) * torch.rand(s["k"].shape[:3], generator=g)
    s["v"].mul_(100)
    s["k"][s["table"][0, 0], 0, 0], s["v"][s["table"][0, 0], 0, 0] = 0, 0
    check(s, 1.0, flushed=2.0 ** -8)


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, HF), (256, BF)])
def test_the_same_requests_in_tables_of_any_width(dim, dtype):
    """What a table row could hold decides over the row tiles, together with all rows: the same requests in rows just
    long enough, and in longer ones, with a workspace of the size that is said to do for every width."""
    new, ctx, hk, page = [50, 37, 64, 1, 0, 61] * 8, [70, 0, 129, 200, 5, 33] * 8, 32, 16
    s = attn_inputs(new, ctx, hk, hk, dim, page, dtype, seed=dim)
    want = dense.attention(s["q"], s["k"], s["v"], s["table"], s["off"], s["ctx"])
    q, off, c, cache = s["q"].cuda(), s["off"].cuda(), s["ctx"].cuda(), B.PagedCache(on_gpu(s["k"]), on_gpu(s["v"]))
    size = B.tree_attention_workspace_bytes(q.shape[0], len(new), hk, cache)
    for keys in (s["table"].shape[1] * page, 320, 336, 512, 1024, 2048, 4096, 4112, 40000):
        if keys < s["table"].shape[1] * page:
            continue
        say("table of", keys, dim, dtype)
        table = torch.full((len(new), keys // page), -1, dtype=torch.int32)
        table[:, :s["table"].shape[1]] = s["table"]
        guard = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        out, lse = B.tree_attention(q, cache, table.cuda(), off, c, return_lse=True, workspace=guard[:size])
        near(out, want[0], want[1], "out")
        near(lse, want[2], want[3], "lse")
        assert bool((guard[size:] == 77).all())


# ---------------------------------------------------------------------------------------------------------------
# row tiles and runs
# ---------------------------------------------------------------------------------------------------------------
def hard_case(new, ctx, hk, grp, dim, page, dtype, words, wide, seed):
    """Requests among which every kind of tile is: pages outside the cache before and after the context's end, in the
    first tiles, and everywhere; rows whose mask leaves nothing; scores that jump by some 25 nats for one row late in a
    request; infinities and NaN in page 0 (which hidden keys are read from), in nobody's pages and past the last keys;
    and in every third request in one new token's values, for the rows that see it."""
    s = attn_inputs(new, ctx, hk * grp, hk, dim, page, dtype, seed=seed, words=words, spare=3)
    r, table = np.random.default_rng(seed), s["table"]
    # page 0 nobody's
    spare = sorted(set(range(s["k"].shape[0])) - set(table[table >= 0].tolist()))[0]
    table[table == 0] = spare
    n_pages = s["k"].shape[0]
    if wide:
        t = torch.full((len(new), wide // page), -1, dtype=torch.int32)
        t[:, :table.shape[1]] = table
        s["table"] = table = t
    bad = [math.nan, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).min]
    for p in set(range(n_pages)) - set(table[table > 0].tolist()):
        for j in range(page):
            s["k"][p, :, j], s["v"][p, :, j] = bad[j % 5], bad[(j + 2) % 5]
    outside = [-1, n_pages, 2 ** 31 - 1, -2 ** 31]
    first = 0
    for i, (m, c) in enumerate(zip(new, ctx)):
        held = -(-(c + m) // page)
        place = lambda j: (int(table[i, j // page]), j % page)  # noqa: E731
        for j in range(c + m, held * page) if i % 2 else ():  # leavings of one request, none of the next
            p, o = place(j)
            s["k"][p, :, o], s["v"][p, :, o] = bad[j % 5], bad[(j + 1) % 5]
        if m and i % 3 == 0:
            p, o = place(c + m // 2)
            s["v"][p, 0, o, 1::4] = [math.inf, math.nan, -math.inf][i // 3 % 3]
        elif m and c > 64:  # for one row, of one head, late
            p, o = place(c - 3)
            row = s["q"][first + m // 2, grp - 1].double()
            s["k"][p, 0, o] = (row * (25 * dim ** 0.5 / row.square().sum())).to(dtype)
        if i % 4 == 1:  # some pages
            for b in r.choice(held, max(1, held // 3), replace=False):
                table[i, b] = outside[int(b) % 4]
        elif i % 8 == 2:  # the first tiles
            table[i, :max(1, held * 2 // 3)] = outside[i % 4]
        elif i % 8 == 6:  # all
            table[i, :held] = outside[i % 4]
        if words and m:
            s["mask"][first + r.choice(m, max(1, m // 5), replace=False)] = 0
        first += m
    return s


def check_hard(s, times=1):
    """times: as often every head, which must give the same bits wherever its runs are."""
    many = dict(s, q=s["q"].repeat(1, times, 1), k=s["k"].repeat(1, times, 1, 1), v=s["v"].repeat(1, times, 1, 1)) if times > 1 else s
    out, lse = attn_run(many)
    assert all(torch.equal(x.nan_to_num(0.0), y.nan_to_num(0.0)) for x, y in zip((out, lse), attn_run(many))), "the same bits again"
    n, hq, dim = s["q"].shape
    assert torch.equal(out.nan_to_num(0.0), out[:, :hq].nan_to_num(0.0).repeat(1, times, 1)) and torch.equal(lse, lse[:, :hq].repeat(1, times))
    out, lse = out[:, :hq], lse[:, :hq]
    o, tol, l, lt = dense.attention(s["q"], s["k"], s["v"], s["table"], s["off"], s["ctx"], s["mask"])
    near(lse, l, lt, "lse")
    assert torch.equal(out.isnan().cpu(), o.isnan()), "NaN where the definition has them"
    near(out.nan_to_num(0.0, math.inf, -math.inf), o.nan_to_num(0.0, math.inf, -math.inf), tol, "out")


FEW = ([40, 7, 33, 52, 61, 20, 48, 30], [0, 290, 300, 130, 77, 1000, 260, 64])
# tokens a request for some 40, 100 and 240 rows by 4 query heads: tiles of 64, of 128 (heads of 128: 256), of 256 (heads of 256: 128)
MANY = {40: [10, 3, 14, 9, 12, 8, 11, 13, 10], 100: [25, 9, 31, 22, 40, 0, 28, 33, 26], 240: [60, 21, 64, 70, 1, 64, 61, 90, 64]}
MANY_CTX = [0, 300, 700, 333, 1025, 260, 512, 40, 500]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("words", [0, 1])
@pytest.mark.parametrize("wide", [0, 5120])
def test_row_tiles_of_several_key_tiles(dim, dtype, words, wide):
    """One key/value head: short row tiles whole, long ones cut into a unit a run; 4 and 1 query heads a group."""
    for grp in (4, 1):
        say("tiles", dim, dtype, words, wide, grp)
        check_hard(hard_case(*FEW, 1, grp, dim, 32, dtype, words, wide, seed=dim + words + grp))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("words", [0, 2])
@pytest.mark.parametrize("rows", [40, 100, 240])
@pytest.mark.parametrize("wide", [0, 5120])
def test_long_runs(wide, rows, dim, dtype, words):
    """Many key/value heads, so that a head has 4 to 8 runs, each over several requests: row tiles' own cost counted in
    units, cut anywhere, and every workgroup's stages and flags used again from one segment to the next."""
    say("runs", wide, rows, dim, dtype, words)
    check_hard(hard_case(MANY[rows], MANY_CTX, 2, 4, dim, 32, dtype, words, wide, seed=rows + dim + words), times=32)


@pytest.mark.parametrize("grp", [33, 64, 65, 100, 128])
@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, HF), (256, BF)])
def test_large_groups(grp, dim, dtype):
    """Up to 128 query heads on a key/value head."""
    for new, ctx, words, wide in (([1, 1, 3, 1, 1], [0, 290, 70, 33, 600], 0, 0), ([5, 9, 2, 7], [40, 0, 300, 99], 1, 0),
                                  ([12, 5, 7], [300, 64, 0], 0, 5120), ([12, 5, 7], [300, 64, 0], 1, 5120)):
        say("groups", grp, dim, dtype, new, words, wide)
        check_hard(hard_case(new, ctx, 2, grp, dim, 32, dtype, words, wide, seed=grp))
