"""Distillation with a tail where the tokens that are not listed lie far below the listed ones, on the GPU, against
log-sums in 64 bits: what the list leaves has a finite loss and a gradient of its own there."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.serving_reference import U32, half_step  # noqa: E402
from tests.test_gpu_scoring import BF, F, HF, hold, many, near  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402

TINY = 2.0 ** -120  # float32's smallest numbers, which an exponential may lose, times a few
GAPS = [0.0, 60.0, 88.0, 90.0, 95.0, 110.0, 200.0, 700.0, 760.0, 1000.0, 10000.0]  # of scale * (listed - others)
RESTS = [0.01, 1e-3, 0.0]  # what the list leaves; 0: what rounding it to float does


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def as_float(scale):
    """What the call takes: 0.7 is off by 2^-25 of itself as a float, which differences of near numbers show."""
    return torch.tensor(scale, dtype=torch.float32).item()


def reference(x, ids, lp, scale, weights):
    """((loss, bound), (dx, bound)) of distill_loss with a tail and the gradient of (weights * loss).sum(), every
    log probability from a difference of log-sums; rows that have listed and other tokens, finite in part.

    A weight exp(scale * (x - max)) is off by 2 + 4 |z - max| half steps (three of its exponent, two of its
    exponential, room for rescaling), the sum of the others' by vocab / 256 + 64 more; the listed ones are in 64 bits, where
    what they leave of 1 keeps 2^-52 for each term."""
    n, v = x.shape
    k, scale = ids.shape[1], as_float(scale)
    z = x.double() * scale
    ids = ids.long()
    there = (ids >= 0) & (ids < v)
    at = ids.clamp(0, v - 1)
    lp = lp.double().masked_fill(~there, -math.inf)
    q = torch.exp(lp)
    mass = q.sum(1, keepdim=True)
    rest = (1 - mass).clamp(min=0)
    listed = torch.zeros(n, v + 1).scatter_(1, torch.where(there, ids, v), 1.0)[:, :v].bool()
    zu = z.masked_fill(listed, -math.inf)
    lse, lse_u = torch.logsumexp(z, 1, keepdim=True), torch.logsumexp(zu, 1, keepdim=True)
    log_pr = lse_u - lse
    log_p = z.gather(1, at) - lse
    terms = torch.where(q > 0, torch.xlogy(q, q) - q * log_p, 0.0)
    size = torch.where(q > 0, q * (lp.abs() + log_p.abs()), 0.0).sum(1, keepdim=True)
    rest_term = torch.where(rest > 0, rest * (torch.log(rest) - log_pr), 0.0)
    loss = terms.sum(1, keepdim=True) + rest_term
    su, p = torch.softmax(zu, 1), torch.softmax(z, 1)  # (of the lowest values a log-sum keeps no count)
    du = (zu - zu.amax(1, keepdim=True)).abs().masked_fill(su == 0, 0)
    rel = U32 * (2 + 4 * (su * du).sum(1, keepdim=True) + v / 256 + 64)
    lost = (k + 16) * 2.0 ** -52  # of what the list leaves
    weight = mass + rest
    loss_tol = (rel * (weight * torch.exp(log_pr) + rest) + torch.where(rest > 0, lost * (2 + torch.log(rest).abs() + log_pr.abs()), 0.0)
                + 1e-13 * (size + rest_term.abs()) + 2 * U32 * loss.abs())
    w = weights.double()[:, None] * scale
    own = torch.zeros(n, v, dtype=torch.float64).scatter_add_(1, at, torch.where(there, q, 0.0))
    dx = w * (weight * p - rest * su * ~listed - own)
    d = (z - z.amax(1, keepdim=True)).abs().masked_fill(p == 0, 0)
    far = torch.where(listed, d, du)
    bound = w.abs() * ((weight * p + rest * su * ~listed) * (U32 * (12 + 4 * far) + rel) + lost * su + U32 * (6 + 2 * k) * own)
    tiny = torch.finfo(x.dtype).tiny * half_step(x.dtype) * 2
    return ((loss[:, 0], loss_tol[:, 0]), (dx, half_step(x.dtype) * dx.abs() + bound * (1 + half_step(x.dtype)) + tiny + TINY * w.abs()))


def rows_of(v, k, dtype, scale, seed):
    """A row for each gap and rest, and one for each rest with the others at the type's lowest value: logits, lists."""
    g = torch.Generator().manual_seed(seed)
    cases = [(gap, rest) for gap in GAPS + [None] for rest in RESTS]
    n = len(cases)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(n)])
    x = torch.randn(n, v, generator=g, dtype=torch.float64)
    for i, (gap, _) in enumerate(cases):
        x[i] = torch.finfo(dtype).min if gap is None else x[i] - gap / scale
        if i % 4 == 1:  # a finite mask: all alike
            x[i] = x[i, 0]
    high = torch.randn(n, k, generator=g, dtype=torch.float64)
    x.scatter_(1, ids, high)
    lp = torch.log_softmax(high * scale + 0.1 * torch.randn(n, k, generator=g, dtype=torch.float64), 1)
    down = torch.full((n, k), -math.inf)
    lp = torch.stack([torch.nextafter(lp[i].float(), down[i]) if rest == 0 else (lp[i] + math.log1p(-rest)).float()
                      for i, (_, rest) in enumerate(cases)])
    if k > 8:  # a list that ends early, and a token named twice: more is left
        ids[5, k - 3:] = -1
        ids[7, 0] = ids[7, 1]
    return x.to(dtype), ids.to(torch.int32), lp, torch.randn(n, generator=g)


def check(x, ids, lp, scale, w, n, offset):
    """The loss by itself, its gradient, both in one call and in place, of rows over and over."""
    loss, dx = reference(x, ids, lp, scale, w)
    assert bool(loss[0].isfinite().all() and dx[0].isfinite().all())
    loss, dx = [tuple(many(t, n) for t in pair) for pair in (loss, dx)]
    dev, a, up = hold(many(x, n), offset, 3), (many(ids, n).cuda(), many(lp, n).cuda()), many(w, n).cuda()
    got = B.distill_loss(dev, *a, tail=True, scale=scale)
    near(got.loss, *loss, "loss")
    near(B.distill_loss_backward(up, dev, *a, got, tail=True, scale=scale), *dx, "dx")
    out = torch.empty(x.shape[1] * n, dtype=x.dtype, device="cuda").view(n, -1)
    both = B.distill_loss(dev, *a, tail=True, scale=scale, weights=up, dlogits=out)
    near(both.loss, *loss, "loss, in one call")
    near(out, *dx, "dx, in one call")
    B.distill_loss(dev, *a, tail=True, scale=scale, weights=up, dlogits=dev)
    assert torch.equal(dev, out)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("scale", [1.0, 10.0])
@pytest.mark.parametrize("n,v,k", [(36, 257, 20), (36, 1280, 100), (36, 9001, 64), (170, 33001, 64), (36, 33001, 256), (170, 70001, 20)])
def test_others_far_below(n, v, k, scale, dtype):
    """By waves and workgroups, in parts, and the one-call form of one, four, eight and sixteen waves."""
    say("far below", n, v, k, scale, dtype)
    x, ids, lp, w = rows_of(v, k, dtype, scale, v + k)
    check(x, ids, lp, scale, w, n, v % 3)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e6])
def test_others_far_above(scale):
    """Listed tokens far below the others: the others' gradient is theirs, the listed ones' is -q."""
    v, k = 5003, 12
    x, ids, lp, w = rows_of(v, k, F, 1.0, 3)
    say("far above", scale)
    check(-x[:33], ids[:33], lp[:33], scale, w[:33], 33, 1)  # (not the lowest value, whose negative is the largest)


def test_gradient_against_differences():
    """Along directions of the other tokens alone, where the loss has no other slope than what the list leaves: with
    weights below e^-90 for them it is linear in their log-sum, whose third derivative is at most 1 for directions of
    entries 1 and -1 times 8; losses of ten are off by a half step, 2^-24 of them, each."""
    n, v, k, h = 4, 301, 12, 2.0 ** -4
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(n, v, generator=g) * 64).round() / 64
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(n)])
    other = torch.ones(n, v).scatter_(1, ids, 0.0)
    x = x - other * torch.tensor([64.0, 96.0, 128.0, 1024.0])[:, None]
    lp = (torch.log_softmax(x.gather(1, ids).double(), 1) + math.log(0.99)).float()
    d = (torch.randint(0, 2, (n, v), generator=g).float() * 2 - 1) * other
    say("differences")
    a = ids.to(torch.int32).cuda(), lp.cuda()
    f = lambda y: B.distill_loss(y.cuda(), *a, tail=True)  # noqa: E731
    slope = (B.distill_loss_backward(torch.ones(n, device="cuda"), x.cuda(), *a, f(x), tail=True).double().cpu() * d).sum(1)
    diff = ((f(x + h * d).loss.double() - f(x - h * d).loss.double()) / (2 * h)).cpu()
    size = f(x).loss.double().cpu().abs() + 1
    assert bool((slope.abs() > 1e-5).all())
    assert bool(((slope - diff).abs() <= 0.01 * 8 * h * h / 6 + size * 2 * U32 / h + v * U32 * 0.01).all()), (slope, diff)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,v,k", [(12, 257, 20), (12, 5003, 64), (12, 33001, 100), (170, 33001, 64), (170, 70001, 256)])
def test_others_of_minus_infinity(n, v, k, dtype):
    """A student under the teacher's own mask, which leaves no token but the listed ones: what rounding leaves of 1 is
    nothing, with all of the list's probability against the student's; what is more than that makes the loss infinite, and
    no gradient of the masked."""
    scale, rests = 0.7, [0.0, 1e-7, 3e-6, 1e-5, 0.01, -1e-7]  # of the list, beside its rounding (-: more than 1)
    g = torch.Generator().manual_seed(v)
    say("minus infinity", n, v, k, dtype)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(12)])
    high = torch.randn(12, k, generator=g).to(dtype)
    x = torch.full((12, v), -math.inf, dtype=dtype).scatter_(1, ids, high)
    lp = torch.log_softmax(high.double() * scale + 0.1 * torch.randn(12, k, generator=g, dtype=torch.float64), 1)
    down = torch.full((k,), -math.inf)
    lp = torch.stack([torch.nextafter(lp[i].float(), down) if i % 6 == 0 else (lp[i] + math.log1p(-rests[i % 6])).float() for i in range(12)])
    scale = as_float(scale)
    q, p, w = torch.exp(lp.double()), torch.softmax(high.double() * scale, 1), torch.randn(12, generator=g)
    mass = q.sum(1, keepdim=True)
    left = 1 - mass
    assert bool((left[::6] > 0).all() and (left[3::6] > 2 ** -18).all() and (left[2::6] < 2 ** -18).all())
    much = left[:, 0] > 2 ** -18
    log_p = torch.log(p)
    loss = (q * (lp.double() - log_p)).sum(1).masked_fill(much, math.inf)
    loss_tol = (q * (lp.abs() + log_p.abs())).sum(1) * 1e-13 + 2 * U32 * loss.abs()
    weight = (mass + left * much[:, None]).clamp(min=0)
    f = w.double()[:, None] * scale
    dx = torch.zeros(12, v, dtype=torch.float64).scatter_(1, ids, f * (weight * p - q))
    d = (high.double() - high.double().amax(1, keepdim=True)).abs() * scale
    bound = torch.zeros(12, v, dtype=torch.float64).scatter_(1, ids, f.abs() * (weight * p * U32 * (8 + 4 * d) + q * 3 * U32))
    bound = half_step(dtype) * dx.abs() + 2 * bound + torch.finfo(dtype).tiny
    dev, a, up = many(x, n).cuda(), (many(ids, n).to(torch.int32).cuda(), many(lp, n).cuda()), many(w, n).cuda()
    got = B.distill_loss(dev, *a, tail=True, scale=scale)
    near(got.loss, many(loss, n), many(loss_tol, n), "loss")
    near(B.distill_loss_backward(up, dev, *a, got, tail=True, scale=scale), many(dx, n), many(bound, n), "dx")
    both = B.distill_loss(dev, *a, tail=True, scale=scale, weights=up, dlogits=dev)
    near(both.loss, many(loss, n), many(loss_tol, n), "loss, in one call")
    near(dev, many(dx, n), many(bound, n), "dx, in one call")


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e20])
@pytest.mark.parametrize("n,v,k", [(36, 257, 20), (36, 9001, 64), (170, 33001, 64)])
def test_scales_at_their_limits(n, v, k, scale):
    """Logits as small, or as large, as the scale makes up for; the type's lowest value among them."""
    say("limits", n, v, k, scale)
    x, ids, lp, w = rows_of(v, k, F, 1.0, v + k)
    keep = 33  # (the lowest value times 1e30 is past the losses' floats)
    check(x[:keep] / torch.tensor(scale), ids[:keep], lp[:keep], scale, w[:keep], n, 1)
