"""Scores of tokens and distillation on the GPU, against plain forms in 64 bits
(tests/scoring_reference.py)."""
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import scoring_reference as ref  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def near(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    ok = (got == want) | torch.where(odd, got.isnan() & want.isnan(), (got - want).abs() <= bound)
    at = (~ok).nonzero()[:1].tolist()
    assert bool(ok.all()), (what, int((~ok).sum()), "values, the first at", at, [float(t[tuple(at[0])]) for t in (got, want, bound)])


def hold(x, offset=0, pad=0):
    """x on the GPU, `offset` elements into its memory, rows `pad` elements longer apart."""
    n, v = x.shape
    store = torch.full((n * (v + pad) + offset,), 3.0, dtype=x.dtype, device="cuda")
    t = store[offset:].view(n, v + pad)[:, :v]
    t.copy_(x)
    return t


def logits(n, v, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, v, generator=g) * spread).to(dtype), g


def check_scores(x, ids, k, scale=1.0, offset=0, pad=0, what="scores"):
    dev = hold(x, offset, pad)
    got = B.token_logprobs(dev, ids.cuda(), top_k=k, scale=scale)
    for name, (want, bound) in ref.scores(x, ids, k, scale).items():
        t = getattr(got, name)
        if bound is None:
            assert torch.equal(t.cpu().long(), want.long()), (what, name, t.cpu(), want)
        else:
            near(t, want, bound, what + " " + name)
    return dev, got


SIZES = [1, 2, 7, 8, 9, 255, 257, 1280, 2051, 8191, 8192, 8193, 33001, 100277]


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("v", SIZES)
def test_scores(v, dtype):
    n = 5
    x, g = logits(n, v, dtype, v)
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[1] = -1
    ids[2] = v if v > 1 else 0
    ids[3] = v - 1
    for k in sorted({0, 1, min(5, v), min(64, v), min(256, v)}):
        say("scores", v, dtype, k)
        check_scores(x, ids, k, scale=[1.0, 0.7][k % 2], offset=k % 5, pad=[0, 3][k % 2])


def many(t, n):
    """Rows of t over and over, n of them."""
    return t[torch.arange(n) % t.shape[0]]


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("v", [513, 1280, 5003, 33001])
@pytest.mark.parametrize("n", [300, 1111, 2200])
def test_scores_of_many_rows(n, v, dtype):
    """Rows in parts and whole ones: each as its like in a small reference."""
    x, g = logits(9, v, dtype, v)
    x[3, 200:] = -INF
    x[4] = -INF
    x[5, 3] = NAN
    x[6] = x[6].round()
    ids = torch.randint(0, v, (9,), generator=g, dtype=torch.int32)
    ids[1] = -1
    for k in (0, 7, 256):
        say("many rows", n, v, dtype, k)
        dev = many(x, n).cuda()
        got = B.token_logprobs(dev, many(ids, n).cuda(), top_k=k)
        for name, (want, bound) in ref.scores(x, ids, k, 1.0).items():
            if bound is None:
                assert torch.equal(getattr(got, name).cpu().long(), many(want, n).long()), name
            else:
                near(getattr(got, name), many(want, n), many(bound, n), name)


@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_rows_with_masks(dtype):
    """Minus infinity and the type's lowest value in masked places, rows with nothing, equal elements, zeros of both
    signs, maxima at either end, NaN and plus infinity: beside ordinary rows, which keep their values."""
    v, k = 9001, 40
    x, g = logits(14, v, dtype, 5)
    low = torch.finfo(dtype).min
    x[1, 100:] = -INF                       # fewer are left than alternatives are asked for: none past them
    x[2, torch.arange(v) % 450 != 7] = -INF  # 20 of them
    x[3] = -INF
    x[4] = low
    x[5, :8990] = low
    x[6] = 0.0
    x[6, ::2] = -0.0
    x[7] = x[7].round()                      # many equal ones
    x[8, 0] = 40.0
    x[9, v - 1] = 40.0
    x[10, 4444] = NAN
    x[11, 17] = INF
    x[12] = -INF
    x[12, 8999] = -3.0
    x[13, 10:] = NAN
    ids = torch.tensor([3, 50, 7, 3, 9000, 8995, 4501, 77, 0, v - 1, 5, 17, 8999, 3], dtype=torch.int32)
    for kk in (0, 1, k, 256):
        say("masks", dtype, kk)
        check_scores(x, ids, kk)
    say("tokens in masked places, and none", dtype)
    ids = torch.tensor([-1, 5000, 8, -5, v, 3, 4500, 78, 1, 0, -1, 18, 0, -1], dtype=torch.int32)
    check_scores(x, ids, k)


@pytest.mark.parametrize("dtype", [BF, F])
def test_alternatives_that_crowd(dtype):
    """Large elements all at places that one thread reads; rising and falling rows; blocks of equal ones."""
    piece = 16 // torch.empty(0, dtype=dtype).element_size()
    v = 1024 * piece * 20 + 5
    x, g = logits(7, v, dtype, 11, spread=1.0)
    group = torch.arange(v) // piece % 1024
    for row, groups in ((0, 1), (1, 2), (2, 255), (3, 20)):
        at = group < groups
        x[row, at] = (10 + torch.randn(int(at.sum()), generator=g)).to(dtype)
    x[4] = torch.linspace(-8, 8, v).to(dtype)
    x[5] = torch.linspace(8, -8, v).to(dtype)
    x[6, 70000:] = 5.0
    ids = torch.tensor([0, 1, 2, 3, v - 1, 100, 70001], dtype=torch.int32)
    for k in (1, 20, 255, 256):
        say("crowd", dtype, k)
        check_scores(x, ids, k)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("v", [1280, 5003, 33001])
def test_alternatives_among_equal_elements(v, dtype):
    """Fewer tokens allowed than alternatives asked for, rows of one value, of two, and of whole numbers: candidates that
    are eight times as many as are wanted, and more."""
    x, g = logits(6, v, dtype, 17)
    x[0, torch.rand(v, generator=g) > 0.005] = -INF
    x[1] = 2.5
    x[2] = (torch.rand(v, generator=g) > 0.5).to(dtype)
    x[3] = x[3].round().clamp(-2, 2)
    x[4, : v // 2] = -INF
    x[4, v // 2:] = 1.0
    x[5] = torch.finfo(dtype).min
    ids = torch.randint(0, v, (6,), generator=g, dtype=torch.int32)
    for k in (1, 16, 64, 65, 200, 256):
        say("equal", v, dtype, k)
        check_scores(x, ids, k)
        n = 1100  # a workgroup or a wave a row
        got = B.token_logprobs(many(x, n).cuda(), many(ids, n).cuda(), top_k=k)
        assert torch.equal(got.top_ids.cpu().long(), many(ref.scores(x, ids, k, 1.0)["top_ids"][0], n))


@pytest.mark.parametrize("dtype,scale", [(BF, 1.0), (HF, 2.0), (F, 0.25), (F, 100.0)])
def test_far_values(dtype, scale):
    """Elements of thousands, and peaks a few units apart."""
    x, g = logits(4, 5003, dtype, 21, spread=1000.0 / scale)
    x[1] = 0.0
    x[2] += 3000.0 / scale
    x[3, 7] = 2000.0 / scale
    say("far", dtype, scale)
    check_scores(x, torch.tensor([1, 2, 3, 7], dtype=torch.int32), 9, scale=scale)


def grads(n, k, g, which):
    t = torch.randn(n, generator=g)
    return dict(g=t if "g" in which else None, gh=torch.randn(n, generator=g) if "h" in which else None,
                gl=torch.randn(n, generator=g) if "l" in which else None, gt=torch.randn(n, k, generator=g) if "t" in which and k else None)


def back_args(up):
    names = dict(g="grad_logprobs", gh="grad_entropy", gl="grad_lse", gt="grad_top")
    return {names[a]: None if t is None else t.cuda() for a, t in up.items()}


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("v,k,which", [(1, 1, "ght"), (7, 3, "g"), (257, 256, "ghlt"), (1280, 5, "h"), (8193, 64, "gt"), (33001, 0, "gl"), (33001, 20, "ghlt"),
                                       (100277, 0, "gh")])
def test_scores_gradient(v, k, which, dtype):
    """Against the formula; into a strided tensor and in place the same bits, and nothing outside the rows."""
    n = 4
    say("scores gradient", v, k, which, dtype)
    x, g = logits(n, v, dtype, v + k)
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    ids[1] = -1
    if v > 20:
        x[2, 5:9] = -INF
    dev, got = check_scores(x, ids, k, 0.8, 1, 2)
    up = grads(n, k, g, which)
    a = back_args(up)
    dx = B.token_logprobs_backward(dev, ids.cuda(), got, **a, scale=0.8)
    near(dx, *ref.scores_grad(x, ids, k, 0.8, **up), "dx")
    store = torch.full((n, v + 5), 7.0, dtype=dtype, device="cuda")
    B.token_logprobs_backward(dev, ids.cuda(), got, **a, scale=0.8, dlogits=store[:, :v])
    assert torch.equal(store[:, :v], dx) and bool((store[:, v:] == 7).all())
    again = B.token_logprobs_backward(dev, ids.cuda(), got, **a, scale=0.8, dlogits=dev)
    assert again is dev and torch.equal(dev, dx)
    if n > 1:
        assert bool((dev.as_strided((n - 1, 2), (v + 2, 1), dev.storage_offset() + v) == 3).all())


def test_gradients_of_odd_rows():
    """Rows with nothing, without probabilities, and without given gradients."""
    v, k, dtype = 1003, 3, F
    x, g = logits(8, v, dtype, 3)
    x[1] = -INF
    x[2, 5] = NAN
    x[3, 5] = NAN
    x[4, 6] = INF
    x[5, 9:] = -INF
    x[6] = torch.finfo(dtype).min
    ids = torch.tensor([1, 2, 3, -1, -1, 700, 5, v + 3], dtype=torch.int32)
    up = grads(8, k, g, "gh")
    up["gh"][3] = 0.0
    say("odd rows")
    dev, got = check_scores(x, ids, k)
    dx = B.token_logprobs_backward(dev, ids.cuda(), got, **back_args(up))
    near(dx, *ref.scores_grad(x, ids, k, 1.0, **up), "dx")
    assert not dx[3].any() and dx[2].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_large_gradients_beside_masked_places(dtype):
    """Given gradients of thousands (a loss scale) where tokens are minus infinity or the type's lowest value."""
    v, k = 1003, 3
    x, g = logits(3, v, dtype, 13)
    x[0, 5:900] = -INF
    x[1, 5:900] = torch.finfo(dtype).min
    ids = torch.tensor([1, 2, 1000], dtype=torch.int32)
    up = {a: None if t is None else t * 4096 for a, t in grads(3, k, g, "ghlt").items()}
    say("large gradients", dtype)
    dev, got = check_scores(x, ids, k, 0.7)
    dx = B.token_logprobs_backward(dev, ids.cuda(), got, **back_args(up), scale=0.7)
    near(dx, *ref.scores_grad(x, ids, k, 0.7, **up), "dx")
    assert not dx[:2, 5:900].any()


def teacher(x, k, g, tail, scale, noise=0.5):
    """Lists of a teacher that differs a little: ids, log probabilities."""
    n, v = x.shape
    t = x.double().clamp(-50, 50) * scale + noise * torch.randn(n, v, generator=g, dtype=torch.float64)
    lp, ids = torch.log_softmax(t, 1).topk(k, 1)
    return ids.to(torch.int32), lp.float() + (0 if tail else 1.5)


def check_distill(x, ids, lp, tail, scale, w, offset=0, pad=0, what="distill"):
    dev = hold(x, offset, pad)
    loss, dx, lse = ref.distill(x, ids, lp, tail, scale, w)
    a = (ids.cuda(), lp.cuda())
    got = B.distill_loss(dev, *a, tail=tail, scale=scale)
    near(got.loss, *loss, what + " loss")
    near(got.lse, *lse, what + " lse")
    d = B.distill_loss_backward(w.cuda(), dev, *a, got, tail=tail, scale=scale)
    near(d, *dx, what + " dx")
    n, v = x.shape
    store = torch.full((n, v + 5), 7.0, dtype=x.dtype, device="cuda")
    both = B.distill_loss(dev, *a, tail=tail, scale=scale, weights=w.cuda(), dlogits=store[:, :v])
    near(both.loss, *loss, what + " loss, in one call")
    near(store[:, :v], *dx, what + " dx, in one call")
    assert bool((store[:, v:] == 7).all())
    B.distill_loss(dev, *a, tail=tail, scale=scale, weights=w.cuda(), dlogits=dev)
    assert torch.equal(dev.nan_to_num(99), store[:, :v].nan_to_num(99))
    return got


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("v,k", [(2, 1), (9, 8), (257, 256), (1280, 16), (8193, 64), (33001, 100), (100277, 64), (140003, 256)])
def test_distill(v, k, dtype):
    n = 4
    x, g = logits(n, v, dtype, v + k)
    w = torch.randn(n, generator=g)
    w[1] = 0.0
    for tail, scale in ((False, 1.0), (True, 1.0), (True, 0.5), (False, 0.5)):
        say("distill", v, k, dtype, tail, scale)
        ids, lp = teacher(x, k, g, tail, scale)
        ids[2, (k + 1) // 2:] = -1  # a list that ends early
        check_distill(x, ids, lp, tail, scale, w, offset=int(tail), pad=3)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("v,k", [(513, 5), (1280, 16), (5003, 64), (33001, 256)])
@pytest.mark.parametrize("n", [300, 1111])
def test_distill_of_many_rows(n, v, k, dtype):
    """Rows in parts and whole ones, loss and gradient apart and in one call: each as its like in a small reference."""
    x, g = logits(7, v, dtype, v)
    w = torch.randn(7, generator=g)
    w[2] = 0.0
    for tail in (False, True):
        say("many rows", n, v, k, dtype, tail)
        ids, lp = teacher(x, k, g, tail, 1.0)
        ids[1] = -1
        y = x.clone()
        y[3] = -INF
        y[4, 5] = NAN
        loss, dx, _ = ref.distill(y, ids, lp, tail, 1.0, w)
        dev, a, up = many(y, n).cuda(), (many(ids, n).cuda(), many(lp, n).cuda()), many(w, n).cuda()
        got = B.distill_loss(dev, *a, tail=tail)
        near(got.loss, many(loss[0], n), many(loss[1], n), "loss")
        near(B.distill_loss_backward(up, dev, *a, got, tail=tail), many(dx[0], n), many(dx[1], n), "dx")
        both = B.distill_loss(dev, *a, tail=tail, weights=up, dlogits=dev)
        near(both.loss, many(loss[0], n), many(loss[1], n), "loss, in one call")
        near(dev, many(dx[0], n), many(dx[1], n), "dx, in one call")


def held_many(x, n, offset):
    return hold(many(x, n), offset)


@pytest.mark.parametrize("n", [160, 512, 513, 1024, 1025])
@pytest.mark.parametrize("pieces,dtype", [(512, BF), (513, F), (1024, BF), (1024, F), (1025, HF)])
def test_on_either_side_of_a_cut(pieces, dtype, n):
    """Counts of rows and of pieces of 16 bytes around which another kernel takes them, rows that begin within a piece."""
    v = pieces * 16 // torch.empty(0, dtype=dtype).element_size()
    x, g = logits(6, v, dtype, pieces)
    x[1] = x[1].round()
    x[2, 50:] = -INF
    ids = torch.randint(0, v, (6,), generator=g, dtype=torch.int32)
    ids[3] = v - 1
    up = torch.randn(6, generator=g)
    for k, offset in ((0, 1), (20, 3), (64, 0)):
        say("cut", n, pieces, dtype, k, offset)
        dev = held_many(x, n, offset)
        got = B.token_logprobs(dev, many(ids, n).cuda(), top_k=k)
        for name, (want, bound) in ref.scores(x, ids, k, 1.0).items():
            if bound is None:
                assert torch.equal(getattr(got, name).cpu().long(), many(want, n).long()), name
            else:
                near(getattr(got, name), many(want, n), many(bound, n), name)
        if k == 0:
            continue
        for tail in (False, True):
            say("distill", tail)
            tops, lp = teacher(x, k, g, tail, 1.0)
            loss, dx, _ = ref.distill(x, tops, lp, tail, 1.0, up)
            a = (many(tops, n).cuda(), many(lp, n).cuda())
            near(B.distill_loss(dev, *a, tail=tail).loss, many(loss[0], n), many(loss[1], n), "loss")
            out = torch.empty_like(dev)
            both = B.distill_loss(dev, *a, tail=tail, weights=many(up, n).cuda(), dlogits=out)
            near(both.loss, many(loss[0], n), many(loss[1], n), "loss, in one call")
            near(out, many(dx[0], n), many(dx[1], n), "dx, in one call")


@pytest.mark.parametrize("v,dtype", [(28672, BF), (28680, BF), (14340, F), (65536, HF), (65544, BF), (32772, F), (4096, F)])
def test_gradients_of_rows_that_fill_their_waves(v, dtype):
    """Loss and gradient in one call at the longest rows of so many waves, and a piece longer."""
    x, g = logits(4, v, dtype, v)
    w = torch.randn(4, generator=g)
    for tail in (False, True):
        say("fill", v, dtype, tail)
        ids, lp = teacher(x, 64, g, tail, 1.0)
        n = 160
        loss, dx, _ = ref.distill(x, ids, lp, tail, 1.0, w)
        out = torch.empty(n, v, dtype=dtype, device="cuda")
        both = B.distill_loss(held_many(x, n, 1), many(ids, n).cuda(), many(lp, n).cuda(), tail=tail, weights=many(w, n).cuda(), dlogits=out)
        near(both.loss, many(loss[0], n), many(loss[1], n), "loss")
        near(out, many(dx[0], n), many(dx[1], n), "dx")


@pytest.mark.parametrize("tail", [False, True])
def test_distill_odd_rows(tail):
    """No teacher, tokens named twice, ids out of range, teachers and students with no probability for a token,
    students with nothing or without probabilities."""
    v, k, dtype = 5003, 6, F
    x, g = logits(13, v, dtype, 8)
    ids, lp = teacher(x, k, g, tail, 1.0)
    ids[1] = -1
    x[1, 3] = NAN
    ids[2, 3] = ids[2, 0]
    ids[2, 5] = ids[2, 0]
    ids[3, 1], ids[3, 2] = v, -7
    lp[4, 2:] = -INF
    x[5, ids[5, 1].long()] = -INF
    x[6, 77] = NAN
    x[7, ids[7, 0].long()] = INF
    x[8] = -INF
    x[9] = torch.finfo(dtype).min
    lp[10] = -INF
    x[11, 100:] = -INF
    ids[11] = torch.arange(6)
    x[12] = -INF  # all that is left is listed
    x[12, ids[12].long()] = 1.0
    w = torch.randn(13, generator=g)
    say("distill odd", tail)
    keep = [i for i in range(13) if not (tail and i == 12)]
    check_distill(x[keep], ids[keep], lp[keep], tail, 1.0, w[keep])
    if tail:
        say("others without any probability where the teacher gives them some")
        got = B.distill_loss(hold(x[12:]), ids[12:].cuda(), lp[12:].cuda(), tail=True)
        assert got.loss.item() == INF


@pytest.mark.parametrize("noise,peak", [(0.0, 0.0), (1e-3, 12.0), (0.5, 30.0)])
def test_distill_near_the_teacher(noise, peak):
    """A tail of almost nothing, and a student that is the teacher: differences of near numbers."""
    v, k = 8193, 20
    x, g = logits(5, v, F, 31)
    x[:, 4000] += peak
    ids, lp = teacher(x, k, g, True, 1.0, noise)
    say("near", noise, peak)
    check_distill(x, ids, lp, True, 1.0, torch.ones(5))


def test_gradient_against_differences():
    """Along random directions d of entries 1 and -1: (f(x + h d) - f(x - h d)) / 2h differs from the derivative by at
    most h^2 / 6 times the third derivative, a third cumulant of numbers up to 1 times 8 or less with its factor, and
    by the losses' own error over h."""
    n, v, k, h = 6, 301, 12, 2.0 ** -6
    x, g = logits(n, v, F, 41, spread=1.0)
    x = (x * 64).round() / 64  # steps are exact
    ids = torch.randint(0, v, (n,), generator=g, dtype=torch.int32)
    t_ids, t_lp = teacher(x, k, g, True, 1.0)
    d = torch.randint(0, 2, (n, v), generator=g).float() * 2 - 1
    dev, dd, one = x.cuda(), d.cuda(), torch.ones(n, device="cuda")
    say("differences")
    for tail in (False, True):
        f = lambda y: B.distill_loss(y, t_ids.cuda(), t_lp.cuda(), tail=tail)  # noqa: E731
        slope = (B.distill_loss_backward(one, dev, t_ids.cuda(), t_lp.cuda(), f(dev), tail=tail).double() * dd).sum(1)
        diff = (f(dev + h * dd).loss.double() - f(dev - h * dd).loss.double()) / (2 * h)
        assert bool(((slope - diff).abs() <= 8 * h * h / 6 + 2 * 1e-5 / h / 2).all()), (tail, slope, diff)
    f = lambda y: B.token_logprobs(y, ids.cuda())  # noqa: E731
    for name, kw in (("logprobs", dict(grad_logprobs=one)), ("entropy", dict(grad_entropy=one)), ("lse", dict(grad_lse=one))):
        slope = (B.token_logprobs_backward(dev, ids.cuda(), f(dev), **kw).double() * dd).sum(1)
        diff = (getattr(f(dev + h * dd), name).double() - getattr(f(dev - h * dd), name).double()) / (2 * h)
        # (an entropy's third derivative has moments of the logarithms too, here up to 10)
        third = 8 * (10 if name == "entropy" else 1)
        assert bool(((slope - diff).abs() <= third * h * h / 6 + 2 * 2e-5 / h / 2).all()), (name, slope, diff)
