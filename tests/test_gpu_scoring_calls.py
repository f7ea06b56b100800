"""Calls of the operators between logits and ids as programs make them: gradients recorded, graphs, streams, given
outputs and workspaces, strides, refusals, and a run of them together."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import scoring_reference as ref  # noqa: E402
from tests.test_gpu_scoring import BF, F, HF, INF, check_scores, hold, logits, many, near, teacher  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def same(a, b):
    return all(torch.equal(x.nan_to_num(7), y.nan_to_num(7)) for x, y in zip(a, b))


# ---- gradients ----
@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_recorded_gradients(dtype):
    """A loss of all differentiable outputs at once, a broadcast gradient, and outputs that are not used."""
    n, v, k = 5, 2051, 4
    say("recorded", dtype)
    x, g = logits(n, v, dtype, 1)
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[2] = -1
    up = dict(g=torch.randn(n, generator=g), gh=torch.randn(n, generator=g), gl=torch.randn(n, generator=g), gt=torch.randn(n, k, generator=g))
    leaf = x.cuda().requires_grad_()
    got = B.token_logprobs(leaf, ids.cuda(), top_k=k, scale=0.8)
    assert got.logprobs.requires_grad and got.top_logprobs.requires_grad and not got.ranks.requires_grad and not got.stats.requires_grad
    torch.autograd.backward([got.logprobs, got.entropy, got.lse, got.top_logprobs], [up[a].cuda() for a in ("g", "gh", "gl", "gt")])
    near(leaf.grad, *ref.scores_grad(x, ids, k, 0.8, **up), "all")
    (d,) = torch.autograd.grad(B.token_logprobs(leaf, ids.cuda()).entropy.sum(), leaf)
    near(d, *ref.scores_grad(x, ids, 0, 1.0, gh=torch.ones(n)), "a sum's")
    say("distillation")
    t_ids, t_lp = teacher(x, 20, g, True, 1.0)
    loss = B.distill_loss(leaf, t_ids.cuda(), t_lp.cuda(), tail=True).loss
    (d,) = torch.autograd.grad(loss.mean(), leaf)
    near(d, *ref.distill(x, t_ids, t_lp, True, 1.0, torch.full((n,), 1.0 / n))[1], "a mean's")


def test_gradients_only_where_wanted():
    n, v = 3, 130
    say("no grad")
    x, g = logits(n, v, F, 2)
    ids, leaf = torch.zeros(n, dtype=torch.int32, device="cuda"), x.cuda().requires_grad_()
    t_ids, t_lp = (t.cuda() for t in teacher(x, 5, g, False, 1.0))
    with torch.no_grad():
        quiet = B.token_logprobs(leaf, ids, top_k=3)
        assert not any(t.requires_grad for t in quiet) and not B.distill_loss(leaf, t_ids, t_lp).loss.requires_grad
    assert same(B.token_logprobs(leaf, ids, top_k=3), quiet) and same(B.token_logprobs(leaf.detach(), ids, top_k=3), quiet)
    say("inputs changed between the passes, and a second derivative, are refused")
    got = B.token_logprobs(leaf, ids)
    loss = B.distill_loss(leaf, t_ids, t_lp).loss
    with torch.no_grad():
        leaf.mul_(2)
    for out in (got.logprobs, loss):
        with pytest.raises(RuntimeError):
            out.sum().backward()
    for out in (B.token_logprobs(leaf, ids).entropy, B.distill_loss(leaf, t_ids, t_lp).loss):
        (d,) = torch.autograd.grad(out.sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            d.sum().backward()
    say("the backward kernels by themselves take inputs that require grad")
    assert not B.token_logprobs_backward(leaf, ids, B.token_logprobs(leaf, ids), quiet.lse).requires_grad
    assert not B.distill_loss_backward(quiet.lse, leaf, t_ids, t_lp, B.distill_loss(leaf, t_ids, t_lp)).requires_grad


# ---- graphs, streams, given outputs ----
@pytest.mark.parametrize("n,v,k", [(3, 33001, 20), (600, 1280, 5), (1100, 5003, 70)])
def test_in_a_graph(n, v, k):
    """Forward and backward captured together and replayed with other inputs, eager calls between; two graphs in turn."""
    say("graph", n, v, k)
    x, g = logits(n, v, BF, 3)
    x, ids = x.cuda(), torch.randint(0, v, (n,), generator=g, dtype=torch.int32).cuda()
    t_ids, t_lp = (t.cuda() for t in teacher(x.cpu()[:4], k, g, True, 1.0))
    t_ids, t_lp = many(t_ids.cpu(), n).cuda(), many(t_lp.cpu(), n).cuda()
    w, up, buf = torch.rand(n, generator=g).cuda(), torch.randn(n, generator=g).cuda(), torch.empty_like(x)

    def step():
        s = B.token_logprobs(x, ids, top_k=k)
        d = B.token_logprobs_backward(x, ids, s, grad_logprobs=up, grad_entropy=w)
        t = B.distill_loss(x, t_ids, t_lp, tail=True)
        e = B.distill_loss_backward(w, x, t_ids, t_lp, t, tail=True)
        B.distill_loss(x, t_ids, t_lp, weights=w, dlogits=buf)
        return list(s) + [d, t.loss, e, buf]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            held.append(step())
    for i in range(4):
        x.mul_(1.125)
        ids.copy_(torch.randint(0, v, (n,), generator=g, dtype=torch.int32))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert same(held[i % 2], want), i


def test_recorded_gradients_in_a_graph():
    say("recorded in a graph")
    n, v, k = 40, 5003, 6
    x, g = logits(n, v, F, 4)
    leaf, ids = x.cuda().requires_grad_(), torch.randint(0, v, (n,), generator=g, dtype=torch.int32).cuda()
    t_ids, t_lp = (t.cuda() for t in teacher(x, k, g, False, 1.0))

    def step():
        s, t = B.token_logprobs(leaf, ids, top_k=k), B.distill_loss(leaf, t_ids, t_lp)
        total = s.logprobs.sum() + s.entropy.mul(0.5).sum() + t.loss.sum()
        return [s.logprobs.detach(), t.loss.detach(), *torch.autograd.grad(total, leaf)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        with torch.no_grad():
            leaf.add_(0.25 * leaf.sin())
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, want)


@pytest.mark.parametrize("n,v", [(2, 33001), (300, 1280), (1100, 5003)])
def test_on_a_stream_and_into_given_outputs(n, v):
    """The same bits on another stream, into given outputs and workspaces; a workspace that is too small is refused."""
    say("stream", n, v)
    k, dt = 9, BF
    x, g = logits(n, v, dt, 5)
    x, ids = x.cuda(), torch.randint(0, v, (n,), generator=g, dtype=torch.int32).cuda()
    t_ids, t_lp = (t.cuda() for t in teacher(x.cpu(), k, g, True, 1.0))
    w = torch.rand(n, generator=g).cuda()
    s, t = B.token_logprobs(x, ids, top_k=k), B.distill_loss(x, t_ids, t_lp, tail=True)
    d, e = B.token_logprobs_backward(x, ids, s, w, w), B.distill_loss_backward(w, x, t_ids, t_lp, t, tail=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    on = dict(stream=side)
    s2, t2 = B.token_logprobs(x, ids, top_k=k, **on), B.distill_loss(x, t_ids, t_lp, tail=True, **on)
    d2 = B.token_logprobs_backward(x, ids, s2, w, w, **on)
    e2 = B.distill_loss_backward(w, x, t_ids, t_lp, t2, tail=True, **on)
    torch.cuda.synchronize()
    assert same(s, s2) and same(t, t2) and torch.equal(d, d2) and torch.equal(e, e2)
    out, out2 = (type(a)(*(torch.zeros_like(b) for b in a)) for a in (s, t))
    room = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    assert B.token_logprobs(x, ids, top_k=k, out=out, workspace=room) is out and same(s, out)
    assert B.distill_loss(x, t_ids, t_lp, tail=True, out=out2, workspace=room) is out2 and same(t, out2)
    if n == 2:
        for call in (lambda: B.token_logprobs(x, ids, top_k=k, workspace=room[:256]), lambda: B.distill_loss(x, t_ids, t_lp, workspace=room[:16]),
                     lambda: B.token_logprobs(x, ids, top_k=k, workspace=room[8:])):
            with pytest.raises(B.BBPEError) as err:
                call()
            assert err.value.status == B.E_WORKSPACE


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with what it allocates itself."""
    say("two streams")
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    xs = [logits(5, 100277, BF, 60 + i)[0].cuda() for i in range(2)]
    ids = torch.arange(5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(B.token_logprobs(xs[i], ids, top_k=20))
    torch.cuda.synchronize()
    for i in (0, 1):
        want = B.token_logprobs(xs[i], ids, top_k=20)
        assert all(same(t, want) for t in got[i])


def test_no_rows_and_broadcast_rows():
    say("no rows")
    x, ids = torch.zeros(0, 50, dtype=BF, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    got = B.token_logprobs(x, ids, top_k=4)
    assert [tuple(t.shape) for t in got] == [(0,)] * 4 + [(0, 4), (0, 4), (0, 2)]
    assert B.token_logprobs_backward(x, ids, got, got.lse).shape == (0, 50)
    top, lp = ids.view(0, 1).expand(0, 3).contiguous(), got.lse.view(0, 1).expand(0, 3).contiguous()
    loss = B.distill_loss(x, top, lp, weights=got.lse, dlogits=x)
    assert loss.loss.shape == (0,) and B.distill_loss_backward(got.lse, x, top, lp, loss).shape == (0, 50)
    say("one row for all")
    y, g = logits(1, 777, F, 6)
    ids = torch.randint(0, 777, (6,), generator=g, dtype=torch.int32)
    wide = B.token_logprobs(y.cuda().expand(6, 777), ids.cuda(), top_k=3)
    for name, (want, bound) in ref.scores(y.expand(6, 777), ids, 3, 1.0).items():
        near(getattr(wide, name), want.double(), 0 if bound is None else bound, name)


def test_rows_far_apart():
    """Rows past 32-bit offsets: 3 rows of 9,001 a billion elements apart; written through as far too."""
    say("far apart")
    n, v, far = 3, 9001, 1 << 30
    x, g = logits(n, v, BF, 7)
    store = torch.zeros(2 * far + v, dtype=BF, device="cuda")
    dev = store.as_strided((n, v), (far, 1))
    dev.copy_(x)
    ids = torch.tensor([5, 9000, 77], dtype=torch.int32)
    got = B.token_logprobs(dev, ids.cuda(), top_k=7)
    near_by = hold(x, pad=7)  # (rows that begin as those do in 16 bytes: sums are added in the same order)
    assert same(got, B.token_logprobs(near_by, ids.cuda(), top_k=7))
    w = torch.rand(n, generator=g).cuda()
    want = B.token_logprobs_backward(near_by, ids.cuda(), got, w, w)
    assert torch.equal(B.token_logprobs_backward(dev, ids.cuda(), got, w, w, dlogits=dev), want)
    assert not store[v:far].any() and not store[far + v:2 * far].any()


def test_gradients_between_the_logits_rows():
    n, v = 40, 5003
    g = torch.Generator(device="cuda").manual_seed(8)
    both = torch.randn(n, 2 * v, generator=g, device="cuda")
    x, dx = both[:, v:], both[:, :v]
    kept, ids = x.clone(), torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(n, generator=g, device="cuda")
    got = B.token_logprobs(x, ids, top_k=6)
    want = B.token_logprobs_backward(x, ids, got, grad_logprobs=w)
    B.token_logprobs_backward(x, ids, got, grad_logprobs=w, dlogits=dx)
    assert torch.equal(dx, want) and torch.equal(x, kept)
    apart = torch.empty_like(kept)
    B.distill_loss(x, got.top_ids, got.top_logprobs, tail=True, weights=w, dlogits=apart)
    B.distill_loss(x, got.top_ids, got.top_logprobs, tail=True, weights=w, dlogits=dx)
    assert torch.equal(x, kept) and bool((dx - apart).abs().max() <= 1e-6)
    with pytest.raises(Exception):
        B.distill_loss(x, got.top_ids, got.top_logprobs, tail=True, weights=w, dlogits=both[:, 1:v + 1])


def test_more_rows_than_a_launch_takes():
    n, v, few = (1 << 21) + 301, 9, 301
    g = torch.Generator().manual_seed(3)
    x = torch.randn(few, v, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, v, (few,), generator=g, dtype=torch.int32)
    lp, tops = torch.log_softmax(x.float(), 1).topk(3, 1)
    w = torch.randn(few, generator=g)
    at = (torch.arange(n) % few).cuda()
    say("few")
    small = [t.cuda() for t in (x, ids, tops.int(), lp, w)]
    large = [t[at] for t in small]

    def run(x, ids, tops, lp, w):
        a = B.token_logprobs(x, ids, top_k=2)
        b = B.distill_loss(x, tops, lp, tail=True)
        out = torch.empty_like(x)
        c = B.distill_loss(x, tops, lp, tail=True, weights=w, dlogits=out)
        return [a.logprobs, a.entropy, a.lse, a.ranks, a.top_ids, a.top_logprobs, b.loss, c.loss, out,
                B.token_logprobs_backward(x, ids, a, grad_logprobs=w), B.distill_loss_backward(w, x, tops, lp, b, tail=True)]

    # (a row's last digits may depend on where it begins in 16 bytes: eight rows of nine elements on, the same)
    want = run(*[t[(torch.arange(8 * few) % few).cuda()] for t in small])
    say("many")
    got = run(*large)
    at = (torch.arange(n) % (8 * few)).cuda()
    for i, (p, q) in enumerate(zip(got, want)):
        assert torch.equal(p, q[at]), i


def test_more_tokens_than_bits_at_a_time():
    """A vocabulary of a million and some: the list's bits are set several times in a row, and places pass 2^20."""
    v, k = 1100003, 100
    say("a million tokens")
    for dtype in (BF, F):
        x, g = logits(2, v, dtype, 8)
        ids = torch.tensor([v - 1, 600000], dtype=torch.int32)
        check_scores(x, ids, k, 0.9)
        t_ids, t_lp = teacher(x, k, g, True, 0.9)
        w = torch.tensor([1.0, -0.5])
        loss, dx, _ = ref.distill(x, t_ids, t_lp, True, 0.9, w)
        for rows in (2, 300):  # in parts, and a workgroup a row
            a = (many(t_ids, rows).cuda(), many(t_lp, rows).cuda())
            dev = many(x, rows).cuda()
            got = B.distill_loss(dev, *a, tail=True, scale=0.9, weights=many(w, rows).cuda(), dlogits=dev)
            near(got.loss, many(loss[0], rows), many(loss[1], rows), "loss")
            near(dev[-2:], *dx, "dx")
            if rows == 2:
                near(B.distill_loss(x.cuda(), *a, tail=True, scale=0.9).loss, *loss, "loss alone")


# ---- refusals ----
def test_refused():
    say("refused")
    n, v, k = 3, 40, 4
    x, ids = torch.zeros(n, v, dtype=BF, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    top, lp, w = torch.zeros(n, k, dtype=torch.int32, device="cuda"), torch.zeros(n, k, device="cuda"), torch.ones(n, device="cuda")
    s, t = B.token_logprobs(x, ids, top_k=k), B.distill_loss(x, top, lp)
    one = torch.zeros(1, v, dtype=BF, device="cuda").expand(n, v)
    for call in (
            lambda: B.token_logprobs(x.double(), ids), lambda: B.token_logprobs(x[0], ids), lambda: B.token_logprobs(x.t(), ids),
            lambda: B.token_logprobs(x, ids.long()), lambda: B.token_logprobs(x, ids[:2]), lambda: B.token_logprobs(x, ids.cpu()),
            lambda: B.token_logprobs(x, ids, top_k=41), lambda: B.token_logprobs(x, ids, top_k=-1), lambda: B.token_logprobs(x, ids, scale=0.0),
            lambda: B.token_logprobs(x, ids, scale=math.nan), lambda: B.token_logprobs(x[:, :0], ids),
            lambda: B.token_logprobs(x, ids, top_k=2, out=s), lambda: B.token_logprobs(torch.zeros(n, 300, device="cuda"), ids, top_k=257),
            lambda: B.token_logprobs_backward(x, ids, s, w.double()), lambda: B.token_logprobs_backward(x, ids, s, w[:2]),
            lambda: B.token_logprobs_backward(x, ids, s, grad_top=w), lambda: B.token_logprobs_backward(x[:2], ids, s, w),
            lambda: B.token_logprobs_backward(x, ids, s, w, dlogits=one), lambda: B.token_logprobs_backward(x, ids, s, w, dlogits=x.float()),
            lambda: B.distill_loss(x, top.long(), lp), lambda: B.distill_loss(x, top, lp.double()), lambda: B.distill_loss(x, top[:, :3], lp),
            lambda: B.distill_loss(x, top[:, :0], lp[:, :0]), lambda: B.distill_loss(x[:, :4], top, lp, tail=True),
            lambda: B.distill_loss(x[:, :3], top, lp), lambda: B.distill_loss(x, top, lp, weights=w, dlogits=one),
            lambda: B.distill_loss(x, top, lp, weights=w[:2], dlogits=x), lambda: B.distill_loss(x, top, lp, scale=-1.0),
            lambda: B.distill_loss_backward(w[:2], x, top, lp, t), lambda: B.distill_loss_backward(w, x, top, lp, t, dlogits=x[:, :39])):
        with pytest.raises(B.BBPEError) as e:
            call()
        assert e.value.status == B.E_INVALID_ARG
    assert B.distill_loss(x[:, :4], top, lp).loss.shape == (n,)


# ---- together ----
def test_teacher_to_student():
    """From a teacher's logits to a student's gradient through both operators, as the definitions in 64 bits have it."""
    n, v, k, scale = 6, 5003, 32, 0.5
    say("teacher to student")
    a, g = logits(n, v, BF, 9)
    b = (a.float() + torch.randn(n, v, generator=g)).to(BF)
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[-1] = -1
    scored = B.token_logprobs(a.cuda(), ids.cuda(), top_k=k, scale=scale)
    want = ref.scores(a, ids, k, scale)
    assert torch.equal(scored.top_ids.cpu().long(), want["top_ids"][0])
    leaf = b.cuda().requires_grad_()
    loss = B.distill_loss(leaf, scored.top_ids, scored.top_logprobs, tail=True, scale=scale).loss
    (d,) = torch.autograd.grad(loss.mean(), leaf)
    l, dx, _ = ref.distill(b, scored.top_ids.cpu(), scored.top_logprobs.cpu(), True, scale, torch.full((n,), 1.0 / n))
    near(loss.detach(), *l, "loss")
    near(d, *dx, "dx")
    say("a student that is the teacher")
    loss = B.distill_loss(a.cuda(), scored.top_ids, scored.top_logprobs, tail=True, scale=scale).loss
    # the lists are rounded to 32 bits, each log probability by half a step: the loss is of second order in that, and
    # the sum of weights' error enters it with what the list leaves
    assert bool((loss.abs() <= ref.distill(a, scored.top_ids.cpu(), scored.top_logprobs.cpu(), True, scale, torch.ones(n))[0][1].cuda() + 1e-12).all())


def test_example():
    """examples/distill_step.py: it runs, and gradients arrive."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_step.py")
    spec = importlib.util.spec_from_file_location("distill_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    scored, losses, leaves = mod.main()
    assert bool(torch.isfinite(scored.logprobs).all()) and all(bool(torch.isfinite(t).all()) for t in losses)
    assert all(bool(torch.isfinite(t.grad).all()) and bool(t.grad.any()) for t in leaves)
