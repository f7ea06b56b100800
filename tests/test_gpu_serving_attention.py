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
