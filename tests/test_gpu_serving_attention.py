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
