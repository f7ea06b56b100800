"""What calls of the operators between ids and attention keep, and refuse, on the GPU, and sizes that
tests/test_gpu_serving.py leaves out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import serving_reference as ref  # noqa: E402
from tests.test_gpu_serving import near, norm_inputs, say, tables_case  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tables_args(tokens, n=2, page=16):
    dev = "cuda"
    off = torch.tensor([0] + [tokens] * n, dtype=torch.int64, device=dev)
    width = -(-tokens // page) + 1
    return (off, torch.zeros(n, dtype=torch.int32, device=dev), torch.arange(width, dtype=torch.int32, device=dev),
            torch.zeros(n, width, dtype=torch.int32, device=dev), page)


@pytest.mark.parametrize("on_a_stream", [False, True])
def test_lengths_do_not_keep_the_tokens_outputs(on_a_stream):
    """seq_len is the next step's ctx_len: what it holds on to is a request's size, not a token's."""
    say("storage", on_a_stream)
    args = tables_args(5000)
    torch.cuda.synchronize()
    plan = B.block_tables(*args, 5000, **(dict(stream=torch.cuda.Stream()) if on_a_stream else {}))
    torch.cuda.synchronize()
    assert plan.seq_len.tolist() == [5000, 0] and plan.wait() == (313, 5000)
    assert max(t.untyped_storage().nbytes() for t in (plan.seq_len, plan.status)) < 1000
    assert all(t.data_ptr() % 16 == 0 for t in plan)


@pytest.mark.parametrize("tokens,page", [(1 << 31, 16), (1 << 40, 16), (1 << 62, 16), (-1, 16), (5, 0), (5, -16), (5, (1 << 30) + 1), (5, 1 << 32)])
def test_sizes_are_refused_before_memory_is_taken(tokens, page):
    say("sizes", tokens, page)
    args = tables_args(5)[:4]
    for kw in ({}, dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(B.BBPEError) as e:
            B.block_tables(*args, page, tokens, **kw)
        assert e.value.status == B.E_INVALID_ARG


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rows_and_weights_16_bytes_off(dtype, inter):
    """Rows, weights and outputs aligned to 16 bytes and to no more, which is all that is asked for."""
    n, hq, hk, dim, eps = 5, 3, 2, 64, 1e-5
    say("16 bytes off", dtype, inter)
    step = 16 // torch.empty(0, dtype=dtype).element_size()
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, dim, dtype, 29)

    def off(shape):  # 16 bytes into an allocation, rows 16 bytes apart besides their elements
        *lead, last = shape
        rows = 1
        for m in lead:
            rows *= m
        store = torch.zeros(rows * (last + step) + step, dtype=dtype, device="cuda")[step:]
        t = store[:rows * (last + step)].view(*lead, last + step)[..., :last]
        assert t.data_ptr() % 32 == 16
        return t
    x, ws = off((n, hq + 2 * hk, dim)), [off((dim,)).copy_(t) for t in w]
    x.copy_(dev)
    q, k = B.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], *ws, pos.cuda(), freq.cuda(), eps=eps, interleaved=inter, q_out=off((n, hq, dim)),
                          k_out=off((n, hk, dim)))
    near(q, *ref.norm_rope(wide[:, :hq], w[0], pos, freq, eps, inter), "q")
    near(k, *ref.norm_rope(wide[:, hq:hq + hk], w[1], pos, freq, eps, inter), "k")
    gq, gk = torch.randn(n, hq, dim, generator=g).to(dtype), torch.randn(n, hk, dim, generator=g).to(dtype)
    gqd, gkd = off((n, hq, dim)).copy_(gq), off((n, hk, dim)).copy_(gk)
    dq, dk, dwq, dwk = B.qk_norm_rope_backward(gqd, gkd, x[:, :hq], x[:, hq:hq + hk], *ws, pos.cuda(), freq.cuda(), eps=eps, interleaved=inter,
                                               dq=off((n, hq, dim)), dk=off((n, hk, dim)))
    for dx, dw, up, xx, ww in ((dq, dwq, gq, wide[:, :hq], w[0]), (dk, dwk, gk, wide[:, hq:hq + hk], w[1])):
        a, b = ref.norm_rope_grad(up, xx, ww, pos, freq, eps, inter)
        near(dx, *a, "dx")
        near(dw, *b, "dw")


@pytest.mark.parametrize("n", [1, 6, 700, 4500])
@pytest.mark.parametrize("before", [1, 3, 300, 5000])
def test_tokens_before_the_first_request(n, before):
    """Offsets that begin above 0: tokens of no request in front, and behind."""
    r = np.random.default_rng(n + before)
    new, ctx = r.integers(0, 40, n), r.integers(0, 90, n)
    say("before the first", n, before)
    off = before + np.concatenate([[0], np.cumsum(new)])
    got, _ = tables_case(new, ctx, 16, q_off=off, n_tokens=int(off[-1]) + 9, depth=bool(n & 1), seed=n)
    assert got.slots[:before].eq(-1).all() and got.requests[:before].eq(-1).all() and got.positions[:before].eq(0).all()


@pytest.mark.parametrize("n,hq,hk,dim,rot,dtype,inter", [(600, 64, 8, 128, 128, torch.bfloat16, False), (1301, 500, 40, 16, 16, torch.float16, True),
                                                         (2100, 40, 40, 96, 32, torch.float32, False), (1030, 20, 20, 256, 128, torch.bfloat16, True)])
def test_norm_of_more_rows_than_a_workgroup_has_at_once(n, hq, hk, dim, rot, dtype, inter):
    """A token's rows in several rounds, forward and backward, with several tokens a batch in the backward pass."""
    say("many heads", n, hq, hk, dim, rot, dtype, inter)
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, rot, dtype, 31)
    args = (dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda(), w[1].cuda(), pos.cuda(), freq.cuda())
    q, k = B.qk_norm_rope(*args, interleaved=inter)
    near(q, *ref.norm_rope(wide[:, :hq], w[0], pos, freq, 1e-6, inter), "q")
    near(k, *ref.norm_rope(wide[:, hq:hq + hk], w[1], pos, freq, 1e-6, inter), "k")
    gq, gk = torch.randn(n, hq, dim, generator=g).to(dtype), torch.randn(n, hk, dim, generator=g).to(dtype)
    got = B.qk_norm_rope_backward(gq.cuda(), gk.cuda(), *args, interleaved=inter)
    for dx, dw, up, x, ww in ((got[0], got[2], gq, wide[:, :hq], w[0]), (got[1], got[3], gk, wide[:, hq:hq + hk], w[1])):
        a, b = ref.norm_rope_grad(up, x, ww, pos, freq, 1e-6, inter)
        near(dx, *a, "dx")
        near(dw, *b, "dw")
    again = B.qk_norm_rope_backward(gq.cuda(), gk.cuda(), *args, interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_norm_of_more_tokens_than_a_launch_takes():
    """2^22 tokens and a few, one head of 16: rows on both sides of the launches' border, and everything else kept."""
    n, dim, at = (1 << 22) + 70, 16, (1 << 22) - 50
    say("many tokens", n)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, 1, dim, generator=g, device="cuda").to(torch.bfloat16)
    w = [torch.ones(dim, dtype=torch.bfloat16, device="cuda") * s for s in (1.5, 0.75)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freq = torch.tensor([1.0, 0.5, 0.25, 0.125, 2e-2, 1e-2, 1e-3, 1e-4], device="cuda")
    q, k = B.qk_norm_rope(x, x, *w, pos, freq)
    for rows in (slice(0, 100), slice(at, n)):
        for got, ww in ((q, w[0]), (k, w[1])):
            near(got[rows], *ref.norm_rope(x[rows].cpu(), ww.cpu(), pos[rows].cpu(), freq.cpu(), 1e-6, False), "rows")
    # the rotation keeps lengths: no row was left out
    assert bool(((q.float().square().mean(-1) - 2.25).abs() < 0.1).all())


def test_outputs_whose_rows_share_memory_are_refused():
    """A broadcast tensor takes one row at last, whichever wrote it."""
    say("shared rows")
    n, hq, hk, dim, dt, dev = 3, 2, 2, 64, torch.bfloat16, "cuda"
    x, one = torch.zeros(n, hq, dim, dtype=dt, device=dev), torch.zeros(1, 1, dim, dtype=dt, device=dev)
    pos, freq = torch.zeros(n, dtype=torch.int32, device=dev), torch.zeros(dim // 2, device=dev)
    cache = B.PagedCache(*(torch.zeros(2, hk, 16, dim, dtype=dt, device=dev) for _ in range(2)))
    attn = (x, cache, torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.tensor([0, n], device=dev), torch.zeros(1, dtype=torch.int32, device=dev))
    for shared in (one.expand(n, hq, dim), torch.zeros(n, 1, dim, dtype=dt, device=dev).expand(n, hq, dim)):
        for call in (lambda: B.qk_norm_rope(x, x, None, None, pos, freq, q_out=shared), lambda: B.qk_norm_rope(x, x, None, None, pos, freq, k_out=shared),
                     lambda: B.qk_norm_rope_backward(x, x, x, x, None, None, pos, freq, dq=shared),
                     lambda: B.qk_norm_rope_backward(x, x, x, x, None, None, pos, freq, dk=shared), lambda: B.tree_attention(*attn, out=shared)):
            with pytest.raises(B.BBPEError) as e:
                call()
            assert e.value.status == B.E_INVALID_ARG and "share memory" in str(e.value)
    # inputs may be broadcast, and a single row has no others
    assert B.qk_norm_rope(one.expand(n, hq, dim), x, None, None, pos, freq)[0].shape == x.shape
    B.qk_norm_rope(one, one, None, None, pos[:1], freq, q_out=one.clone().expand(1, 1, dim))
    with pytest.raises(B.BBPEError):
        B.qk_norm_rope(x, x, None, None, pos, torch.tensor(1.0, device=dev))
