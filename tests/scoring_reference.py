"""Plain forms, in 64 bits on the CPU, of the operators between logits and ids
(byte_level_bpe_amd/scoring.py), with the error that 32-bit arithmetic and one
rounding to the output's type can make."""
import math

import torch

from tests.serving_reference import U32, half_step

TINY = 2.0 ** -120  # float32's smallest numbers, which an exponential may lose, times a few


class Row:
    """Softmax of rows z = scale * x, and what 32 bits may be off by.

    A weight's exponent is off by three half steps of itself (the difference, the factor, the product), the weight by
    two more (its exponential): 2 + 4 |z - max| half steps with room for its rescaling.  The sum over a thread's
    elements, waves and workgroups adds a half step each time: under vocab / 256 + 64 of them."""

    def __init__(self, x, scale):
        self.z = x.double() * scale
        self.bad = ~(x.double() < math.inf).all(1)  # a NaN or plus infinity
        top = self.z.amax(1, keepdim=True)
        self.none = (top == -math.inf).squeeze(1)
        self.top = top.masked_fill(~torch.isfinite(top), 0)
        self.d = self.z - self.top
        self.p = torch.softmax(self.z.masked_fill((self.none | self.bad)[:, None], 0), 1).masked_fill(self.none[:, None], 0)
        self.log_sum = torch.log(torch.exp(self.d).sum(1, keepdim=True))
        self.lse = self.top + self.log_sum
        self.logp = (self.d - self.log_sum).masked_fill(self.none[:, None], -math.inf)
        self.d0 = self.d.masked_fill(self.p == 0, 0)
        self.far = (self.p * self.d0.abs()).sum(1, keepdim=True)
        far2 = (self.p * self.d0 ** 2).sum(1, keepdim=True)
        steps = x.shape[1] / 256 + 64
        self.rel = U32 * (2 + 4 * self.far + steps)          # of the sum of weights
        self.rel_mean = U32 * ((2 + steps) * self.far + 4 * far2) + self.far * self.rel  # of E[max - z]
        self.entropy = -(self.p * self.logp.masked_fill(self.p == 0, 0)).sum(1, keepdim=True)
        self.entropy_tol = self.rel + self.rel_mean + 2 * U32 * (self.entropy.abs() + self.log_sum.abs())

    def weight_tol(self):
        """Of p_j, relative: its exponent and exponential, the sum, and its logarithm kept in 32 bits."""
        return U32 * (4 + 4 * self.d0.abs() + 3 * self.log_sum.abs()) + self.rel


def scores(x, ids, k, scale):
    """{name: (value, bound)}: token_logprobs; whole numbers with bound None."""
    r, n, v = Row(x, scale), x.shape[0], x.shape[1]
    ids = ids.long()
    given, far = (ids >= 0) & (ids < v), ids >= v
    bad = r.bad[:, None]
    at = ids.clamp(0, v - 1)[:, None]
    tol = lambda value: r.rel + 2 * U32 * (value.abs().masked_fill(value.isinf(), 0) + r.log_sum.abs())  # noqa: E731
    lp = r.logp.gather(1, at)
    lp_tol = tol(lp)
    lp = lp.masked_fill(bad, math.nan)
    lp = torch.where(given[:, None], lp, torch.where(far[:, None], math.nan, 0.0))
    first = torch.sort(x.double() + 0.0, dim=1, descending=True, stable=True).indices
    ranks = torch.argsort(first, dim=1).gather(1, at)[:, 0] + 1
    top = first[:, :k]
    top_lp = r.logp.gather(1, top)
    entropy = r.entropy.masked_fill(r.none[:, None], 0).masked_fill(bad, math.nan)
    lse = r.lse.masked_fill(r.none[:, None], -math.inf)
    one = lambda t: t[:, 0]  # noqa: E731
    return {
        "logprobs": (one(lp), one(lp_tol)), "entropy": (one(entropy), one(r.entropy_tol)),
        "lse": (one(lse.masked_fill(bad, math.nan)), one(tol(r.lse))),
        "ranks": (torch.where(given & ~r.bad, ranks, 0), None), "top_ids": (top.masked_fill(bad, -1), None),
        "top_logprobs": (top_lp.masked_fill(bad, math.nan), tol(top_lp)),
    }


def scores_grad(x, ids, k, scale, g=None, gh=None, gl=None, gt=None):
    """(dx, bound): gradient of sum g logprob + gh entropy + gl lse + gt . top_logprobs."""
    r, n, v = Row(x, scale), x.shape[0], x.shape[1]
    zero = torch.zeros(n, 1, dtype=torch.float64)
    col = lambda t: zero if t is None else t.double()[:, None]  # noqa: E731
    ids = ids.long()[:, None]
    given = (ids >= 0) & (ids < v)
    g, gh, gl = col(g) * given, col(gh), col(gl)
    gt = torch.zeros(n, k, dtype=torch.float64) if gt is None else gt.double()
    top = torch.sort(x.double() + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    own = torch.zeros(n, v, dtype=torch.float64)
    own.scatter_add_(1, ids.clamp(0, v - 1), g)
    size = torch.zeros_like(own)
    size.scatter_add_(1, ids.clamp(0, v - 1), g.abs())
    own.scatter_add_(1, top, gt)
    size.scatter_add_(1, top, gt.abs())
    all_g = g + gt.sum(1, keepdim=True) - gl
    logp = r.logp.masked_fill(r.p == 0, 0)
    dx = scale * (own - r.p * (all_g + gh * (logp + r.entropy)))
    mass = g.abs() + gt.abs().sum(1, keepdim=True) + gl.abs()
    inner = mass + gh.abs() * (r.d0.abs() + 2 * r.log_sum.abs() + r.entropy)
    bound = scale * (r.p * (inner * (r.weight_tol() + (16 + k) * U32) + gh.abs() * r.entropy_tol) + (8 + k) * U32 * size)
    # with no gradient given, a row's is 0 whatever it holds; with nothing in the row there is none
    quiet = ((mass == 0) & (gh == 0)).squeeze(1) | r.none
    dx = dx.masked_fill(r.bad[:, None], math.nan).masked_fill(quiet[:, None], 0)
    tiny = torch.finfo(x.dtype).tiny * half_step(x.dtype) * 2
    return dx, half_step(x.dtype) * dx.abs() + bound * (1 + half_step(x.dtype)) + tiny + TINY * (inner + size) * scale


def distill(x, ids, lp, tail, scale, weights):
    """((loss, bound), (dx, bound), (lse, bound)): distill_loss, and the gradient of (weights * loss).sum()."""
    r, n, v = Row(x, scale), x.shape[0], x.shape[1]
    ids = ids.long()
    there = (ids >= 0) & (ids < v)
    lp = lp.double().masked_fill(~there, -math.inf)
    q = torch.exp(lp)
    mass = q.sum(1, keepdim=True)
    teacher = there.any(1) if tail else (lp > -math.inf).any(1)
    if not tail:
        q = torch.softmax(lp.masked_fill(~teacher[:, None], 0), 1).masked_fill(~teacher[:, None], 0)
        mass = q.sum(1, keepdim=True)
    rest = (1 - mass).clamp(min=0) if tail else torch.zeros(n, 1, dtype=torch.float64)
    at = ids.clamp(0, v - 1)
    logp = r.logp.gather(1, at)
    some = q > 0
    terms = torch.where(some, torch.xlogy(q, q) - q * logp, 0.0)
    listed = torch.zeros(n, v + 1).scatter_(1, torch.where(there, ids, v), 1.0)[:, :v].bool()
    p_listed = (r.p * listed).sum(1, keepdim=True)
    p_rest = (r.p * ~listed).sum(1, keepdim=True)
    log_rest = torch.log(p_rest)
    rel = r.rel
    if tail:  # the sum is over the others, relative to their own largest
        far = (r.p * ~listed * (r.d0 - r.d0.masked_fill(listed, -math.inf).amax(1, keepdim=True).clamp(min=-1e30)).abs()).sum(1, keepdim=True)
        rel = torch.maximum(rel, U32 * (2 + 4 * far / p_rest.clamp(min=1e-300) + v / 256 + 64))
    rest_term = torch.where(rest > 0, torch.xlogy(rest, rest) - rest * log_rest, 0.0)
    loss = terms.sum(1, keepdim=True) + rest_term
    # the sum of weights is off by r.rel in every log p; log p_rest by the listed share of that
    loss_tol = mass * (rel + 1e-12) + rest * (rel + 1e-12) * p_listed + 2 * U32 * loss.abs().masked_fill(~loss.isfinite(), 0) + 1e-30
    share = torch.where(rest > 0, rest / p_rest, 0.0).masked_fill(p_rest == 0, 0)
    weight = mass + rest if tail else teacher[:, None].double()
    own = torch.zeros(n, v, dtype=torch.float64).scatter_add_(1, at, torch.where(there, q, 0.0))
    own_size = torch.zeros(n, v, dtype=torch.float64).scatter_add_(1, at, torch.where(there, q * (1 + lp.abs().masked_fill(lp.isinf(), 0)), 0.0))
    w = weights.double()[:, None] * scale
    dx = w * (r.p * (weight - share * ~listed) - own)
    factor = (weight - share * ~listed).abs()
    # factor: 64 bits but for the sum of weights, rounded once; q: its exponent in 32 bits (the list's sum too)
    bound = w.abs() * (r.p * (factor * ((r.weight_tol() + rel) + 8 * U32) + share * ~listed * 2 * rel) + U32 * (12 + 2 * ids.shape[1]) * own_size)
    quiet = ~teacher | (weights == 0)
    dx = dx.masked_fill(r.bad[:, None], math.nan).masked_fill((quiet | r.none)[:, None], 0)
    loss = loss.masked_fill(r.none[:, None], math.inf).masked_fill(r.bad[:, None], math.nan).masked_fill(~teacher[:, None], 0)
    tiny = torch.finfo(x.dtype).tiny * half_step(x.dtype) * 2
    lse = r.lse.masked_fill(r.none[:, None], -math.inf).masked_fill(r.bad[:, None], math.nan)
    return ((loss[:, 0], loss_tol[:, 0]),
            (dx, half_step(x.dtype) * dx.abs() + bound * (1 + half_step(x.dtype)) + tiny + TINY * w.abs()),
            (lse[:, 0], (rel + 2 * U32 * (r.lse.abs() + r.log_sum.abs()))[:, 0]))
