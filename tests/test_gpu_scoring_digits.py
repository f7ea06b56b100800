"""Digits of what the operators between logits and ids make, on the GPU: rows whose sums of weights are exact, or a 1 and
many small ones, so that results are off by what their last few operations round; and scales at their limits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.serving_reference import U32  # noqa: E402
from tests import scoring_reference as ref  # noqa: E402
from tests.test_gpu_scoring import F, logits, many, near  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402

SIZES = [300, 1280, 5003, 33001, 50257, 100277, 200005]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def flat(v):
    """Rows of one value, of one value in every third place, and of one value up to the middle: weights are 1 or 0."""
    x = torch.full((3, v), 0.5)
    x[1, torch.arange(v) % 3 != 0] = -math.inf
    x[2, v // 2:] = -math.inf
    return x, torch.exp(x.double() - 0.5) / torch.exp(x.double() - 0.5).sum(1, keepdim=True)


@pytest.mark.parametrize("v", SIZES)
def test_probabilities_in_the_scores_gradient(v):
    """The log-sum's gradient is p: one over the sum, rounded once, times 1.  The entropy's is 0 where all that can
    come is alike: of log p + entropy, two numbers up to 13 that are a half step off each, three with their sum."""
    say("scores", v)
    x, p = flat(v)
    dev, ids = x.cuda(), torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda")
    got, one = B.token_logprobs(dev, ids), torch.ones(3, device="cuda")
    near(B.token_logprobs_backward(dev, ids, got, grad_lse=one), p, 2 * U32 * p, "p")
    near(B.token_logprobs_backward(dev, ids, got, grad_entropy=one), 0 * p, 4 * U32 * 13 * p, "entropy")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", SIZES)
def test_probabilities_in_the_distillation_gradient(v, tail):
    """Where a token is not listed the gradient is p (times what p_r and the list's remainder make of it): a factor in
    64 bits, rounded once, times 1."""
    say("distillation", v, tail)
    x, p = flat(v)
    dev = x.cuda()
    ids = torch.tensor([[0, 3, 6, 9]] * 3, dtype=torch.int32)
    lp = torch.full((3, 4), math.log(0.125))
    other = torch.ones(3, v).scatter_(1, ids.long(), 0.0).double()
    mass = torch.exp(lp.double()).sum(1, keepdim=True)
    want = p * (1 - (1 - mass) / (p * other).sum(1, keepdim=True)) * other if tail else p * other
    a, one = (ids.cuda(), lp.cuda()), torch.ones(3, device="cuda")
    apart = B.distill_loss_backward(one, dev, *a, B.distill_loss(dev, *a, tail=tail), tail=tail)
    both = torch.empty_like(dev)
    B.distill_loss(dev, *a, tail=tail, weights=one, dlogits=both)
    for got, what in ((apart, "apart"), (both, "in one call")):
        near(got.cpu().double() * other, want, 2 * U32 * want.abs(), what)


@pytest.mark.parametrize("offset", [0.0, 1.5, 300.0, -1e3, 1e4, -1e4, 1e5])
@pytest.mark.parametrize("v,k", [(300, 5), (1280, 100), (33001, 256)])
def test_lists_with_a_constant_added(v, k, offset):
    """Without a tail a list is made to sum to 1, whatever is added to all of a row.  Listed tokens get p - q: each of the
    two is in 64 bits and rounded once, then their difference; no bound of the offset, nor of the list's length."""
    say("constant added", v, k, offset)
    x, p = flat(v)
    g = torch.Generator().manual_seed(v + k)
    ids = torch.stack([torch.randperm(v, generator=g)[:k] for _ in range(3)]).to(torch.int32)
    lp = (torch.randn(3, k, generator=g) + offset).float()
    q = torch.softmax(lp.double(), 1)
    want = p.scatter_add(1, ids.long(), -q)
    size = p.scatter_add(1, ids.long(), q)
    dev, a, one = x.cuda(), (ids.cuda(), lp.cuda()), torch.ones(3, device="cuda")
    apart = B.distill_loss_backward(one, dev, *a, B.distill_loss(dev, *a))
    both = torch.empty_like(dev)
    B.distill_loss(dev, *a, weights=one, dlogits=both)
    for got, what in ((apart, "apart"), (both, "in one call")):
        near(got, want, 3 * U32 * size, what)


@pytest.mark.parametrize("n,v", [(6, 300), (6, 5003), (6, 33001), (1200, 9001)])
def test_gradient_of_alternatives_without_probabilities(n, v):
    """A row with a NaN or plus infinity has NaN for its alternatives' log probabilities, and no ids: where a gradient comes
    back to them alone, the row's is NaN; where zeros do, it is 0, and beside them rows keep theirs."""
    say("no probabilities", n, v)
    x = torch.randn(6, v, generator=torch.Generator().manual_seed(v))
    x[1, 7] = x[2, v - 1] = math.nan
    x[3, 5] = math.inf
    rows = torch.arange(n) % 6
    dev, ids = x[rows].cuda(), torch.full((n,), -1, dtype=torch.int32, device="cuda")
    g = torch.zeros(6, 4)
    g[0], g[1], g[3, 2], g[4, 0] = 1.0, 0.5, 1.0, -2.0
    got = B.token_logprobs(dev, ids, top_k=4)
    dx = B.token_logprobs_backward(dev, ids, got, grad_top=g[rows].cuda()).cpu()
    odd = (rows == 1) | (rows == 3)
    assert bool(dx[odd].isnan().all()) and bool(dx[~odd].isfinite().all()) and not dx[(rows == 2) | (rows == 5)].any()
    p = torch.softmax(x.double(), 1)
    for row in (0, 4):
        want = -p[row] * g[row].sum()
        want[got.top_ids[row].cpu().long()] += g[row]
        # the terms, their sum and p's: a few half steps each; its weights' exponents up to 4 |z - max| more
        bound = U32 * (p[row] * g[row].abs().sum() * (16 + 4 * (x[row] - x[row].max()).abs() + v / 256 + 64) + 8 * want.abs())
        assert bool(((dx[row] - want).abs() <= bound).all())


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F])
@pytest.mark.parametrize("n,v", [(16, 1280), (16, 4001), (16, 9001), (16, 33001), (1040, 9001), (600, 33001)])
def test_losses_of_few_digits(n, v, dtype, tail):
    """One token far above all others, which are alike, and listed: the loss is log(1 + (v - 1) e^-d), a tenth or so.

    Each thread's sum is brought to the row's maximum by one factor, off by three half steps (its exponential's two, and
    less than one of an exponent up to a half); the largest element's own piece is added in three roundings beside 1,
    and its thread's other elements, one in 64 or fewer, are off by what their exponents up to 32 are, 24 half steps; the
    loss is rounded once."""
    say("few digits", n, v, dtype, tail)
    d = math.log(10 * v) + torch.arange(16) * 0.13
    x = torch.zeros(16, v).copy_(-d[:, None]).to(dtype)
    top = (torch.arange(16) * 997) % v
    x[torch.arange(16), top] = 0.0
    others = (v - 1) * torch.exp(x.double().amin(1))
    want = torch.log1p(others)
    # (with a tail the list's one probability is 1: nothing is left)
    rows = torch.arange(n) % 16
    a = top.to(torch.int32)[rows, None].cuda(), torch.zeros(n, 1, device="cuda")
    bound = U32 * (3 + others * (3 + 24 / 64) + want) + 1e-12
    dev, w = x[rows].cuda(), torch.ones(n, device="cuda")
    near(B.distill_loss(dev, *a, tail=tail).loss, want[rows], bound[rows], "loss")
    near(B.distill_loss(dev, *a, tail=tail, weights=w, dlogits=torch.empty_like(dev)).loss, want[rows], bound[rows], "in one call")


@pytest.mark.parametrize("k", [0, 5, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F])
@pytest.mark.parametrize("n,v", [(16, 1280), (16, 4001), (16, 9001), (16, 33001), (1040, 9001), (600, 33001)])
def test_scores_of_likely_tokens(n, v, dtype, k):
    """The same rows: the likely token's log probability is -log(1 + (v - 1) e^-d), a tenth or so, with the same bound."""
    say("likely tokens", n, v, dtype, k)
    d = math.log(10 * v) + torch.arange(16) * 0.13
    x = torch.zeros(16, v).copy_(-d[:, None]).to(dtype)
    top = (torch.arange(16) * 997) % v
    x[torch.arange(16), top] = 0.0
    others = (v - 1) * torch.exp(x.double().amin(1))
    want = -torch.log1p(others)
    rows = torch.arange(n) % 16
    bound = U32 * (3 + others * (3 + 24 / 64) - want) + 1e-12
    got = B.token_logprobs(x[rows].cuda(), top.to(torch.int32)[rows].cuda(), top_k=k)
    near(got.logprobs, want[rows], bound[rows], "logprobs")
    near(got.lse, -want[rows], bound[rows], "lse")
    if k:
        near(got.top_logprobs[:, 0].contiguous(), want[rows], bound[rows], "top")


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-3, 1e20])
@pytest.mark.parametrize("n,v", [(5, 300), (5, 33001), (600, 9001)])
def test_scores_at_the_scales_limits(n, v, scale):
    """Logits as small, or as large, as the scale makes up for, with the gradient of every output."""
    say("limits", n, v, scale)
    x, g = logits(5, v, F, v)
    x[1, 5:40] = -math.inf
    x[2] = x[2].round()
    x = x / torch.tensor(scale)
    ids = torch.randint(0, v, (5,), generator=g, dtype=torch.int32)
    up = dict(g=torch.randn(5, generator=g), gh=torch.randn(5, generator=g), gl=torch.randn(5, generator=g), gt=torch.randn(5, 20, generator=g))
    as_float = torch.tensor(scale, dtype=torch.float32).item()
    dev, there = many(x, n).cuda(), many(ids, n).cuda()
    got = B.token_logprobs(dev, there, top_k=20, scale=scale)
    for name, (want, bound) in ref.scores(x, ids, 20, as_float).items():
        if bound is None:
            assert torch.equal(getattr(got, name).cpu().long(), many(want, n).long()), name
        else:
            near(getattr(got, name), many(want, n), many(bound, n), name)
    args = {name: many(up[a], n).cuda() for a, name in (("g", "grad_logprobs"), ("gh", "grad_entropy"), ("gl", "grad_lse"), ("gt", "grad_top"))}
    dx = B.token_logprobs_backward(dev, there, got, **args, scale=scale)
    want, bound = ref.scores_grad(x, ids, 20, as_float, **up)
    near(dx, many(want, n), many(bound, n), "dx")
