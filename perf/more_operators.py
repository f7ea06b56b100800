"""What is measured of the operators between a model's logits and ids: scores of tokens, and distillation.

  token_logprobs   log probabilities of given tokens with entropy, rank and top alternatives, and its backward pass
  distill_loss     divergence from a teacher's top log probabilities, and its gradient

Sizes: vocabularies are those of this repository's tables (1,280 tokens; 100,256 with five specials, ids up to
100,276; 200,000 with five specials, ids up to 200,004) and generic ones; rows are the tokens of a step, a prompt or a
training batch.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's sampled token with its alternatives, the small table: the launch is all it costs
        dict(name="scores one", op="scores", form="forward", dtype="f32", rows=1, vocab=1280, k=20, mask="none", temp=1.0),
        # a decode step of a small batch, a vocabulary of an odd size, so that rows have every alignment
        dict(name="scores step", op="scores", form="forward", dtype="bf16", rows=8, vocab=100277, k=5, mask="none", temp=0.8),
        # a decode step of a large batch, a grammar that leaves few tokens of the large table
        dict(name="scores batch", op="scores", form="forward", dtype="f32", rows=128, vocab=200005, k=20, mask="allowed", temp=1.0),
        # prompts scored: the perplexity of 8,192 tokens
        dict(name="scores prompt", op="scores", form="forward", dtype="bf16", rows=8192, vocab=100277, k=0, mask="none", temp=1.0),
        # a teacher's side of distillation: 64 alternatives of each token, embedding rows padded to a multiple of 64
        dict(name="scores teacher", op="scores", form="forward", dtype="bf16", rows=4096, vocab=200064, k=64, mask="pad", temp=1.5),
        # a policy's training step: log probabilities and entropies with their gradient
        dict(name="scores gradient", op="scores", form="gradient", dtype="bf16", rows=4096, vocab=100277, k=0, mask="none", temp=1.0),
        # the same, small and odd
        dict(name="scores gradient odd", op="scores", form="gradient", dtype="f16", rows=777, vocab=5003, k=0, mask="pad", temp=0.7),
        # distillation with the small table, short lists: a step of a small model
        dict(name="distill small", op="distill", form="gradient", dtype="f32", rows=64, vocab=1280, k=16, tail=False, temp=1.0),
        # the loss by itself on held-out text
        dict(name="distill evaluation", op="distill", form="loss", dtype="bf16", rows=2048, vocab=200005, k=20, tail=True, temp=1.0),
        # a training step: loss, then gradient, with what the teacher's list leaves out as one more outcome
        dict(name="distill gradient", op="distill", form="gradient", dtype="bf16", rows=4096, vocab=100277, k=64, tail=True, temp=2.0),
        # loss and gradient in one call, long lists, logits in 32 bits
        dict(name="distill step", op="distill", form="step", dtype="f32", rows=2048, vocab=200005, k=256, tail=False, temp=1.0),
        # the same in 16 bits over an odd count of rows
        dict(name="distill step odd", op="distill", form="step", dtype="f16", rows=1111, vocab=50021, k=50, tail=True, temp=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, dtype = rng.choice(["scores", "distill"]), rng.choice(["bf16", "bf16", "f16", "f32"])
    vocab = rng.choice([1280, 100256, 100277, 200005, 200064, _log(rng, 300, 260000), _log(rng, 300, 260000), _log(rng, 300, 260000)])
    rows = _log(rng, 1, 8192)
    while rows * vocab * (2 if dtype == "f32" else 1) > 8e8:
        rows -= rows // 3
    k, temp = _log(rng, 1, 256), rng.choice([1.0, 1.0, 0.7, 1.3, 2.0])
    if op == "scores":
        form = rng.choice(["forward", "forward", "gradient"])
        return dict(op=op, form=form, dtype=dtype, rows=rows, vocab=vocab, k=0 if form == "gradient" or rng.random() < 0.25 else k, mask=rng.choice(["none", "none", "pad", "allowed"]), temp=temp)
    return dict(op=op, form=rng.choice(["loss", "gradient", "step"]), dtype=dtype, rows=rows, vocab=vocab, k=k, tail=rng.random() < 0.5, temp=temp)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return _prepare_scores(case, g) if case["op"] == "scores" else _prepare_distill(case, g)


def _logits(case, g):
    """A model's: a wide body, and eight tokens a row that stand out."""
    n, v, t = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    x = torch.randn(n, v, generator=g, device=DEV, dtype=t).mul_(2)
    peaks = torch.randint(0, v, (n, 8), generator=g, device=DEV)
    x.scatter_reduce_(1, peaks, (6 + 8 * torch.rand(n, 8, generator=g, device=DEV)).to(t), "amax")
    return x, peaks


def _upstream(case):
    """A mean's gradient; in float16 with a loss scale, without which most of it would vanish."""
    return (1024.0 if case["dtype"] == "f16" else 1.0) / case["rows"]


def _prepare_scores(case, g):
    n, v = case["rows"], case["vocab"]
    x, peaks = _logits(case, g)
    # given tokens: mostly likely ones, some others; the last of each request has none
    pick = torch.rand(n, generator=g, device=DEV)
    ids = torch.where(pick < 0.7, peaks[:, 0], torch.randint(0, v, (n,), generator=g, device=DEV))
    if case["mask"] == "pad":
        x[:, v - v // 50:] = -math.inf
    if case["mask"] == "allowed":  # a few hundred tokens of a large table, the given one among them
        shut = torch.rand(1, v, generator=g, device=DEV) * 200 > 1
        shut = shut.expand(n, v).clone().scatter_(1, ids[:, None], False)
        x.masked_fill_(shut, -math.inf)
    ids = torch.where((pick > 0.98) & (n > 1), -1, ids).to(torch.int32)
    s = dict(case=case, logits=x, ids=ids, scale=1 / case["temp"])
    if case["form"] == "gradient":
        s["g_logprobs"] = torch.randn(n, generator=g, device=DEV) * _upstream(case)
        s["g_entropy"] = torch.randn(n, generator=g, device=DEV) * 0.1 * _upstream(case)
    return s


def _prepare_distill(case, g):
    n, v, k = case["rows"], case["vocab"], min(case["k"], case["vocab"] - 1)
    x, _ = _logits(case, g)
    # the teacher agrees by and large
    teacher = torch.randn(n, v, generator=g, device=DEV).add_(x).mul_(1 / case["temp"])
    lse = torch.logsumexp(teacher, dim=1, keepdim=True)
    values, ids = torch.topk(teacher, k, dim=1)
    top = values - lse
    # one list in four ends early, and a few rows have none (padding)
    length = torch.where(torch.rand(n, 1, generator=g, device=DEV) < 0.25, torch.randint(1, k + 1, (n, 1), generator=g, device=DEV), k)
    length = torch.where(torch.rand(n, 1, generator=g, device=DEV) < 0.03, 0, length)
    out = torch.arange(k, device=DEV)[None, :] >= length
    s = dict(case=case, logits=x, top_ids=ids.masked_fill(out, -1).to(torch.int32), top=top.masked_fill(out, -math.inf), scale=1 / case["temp"])
    if case["form"] != "loss":
        s["weights"] = torch.where(length[:, 0] > 0, _upstream(case), 0.0)
    if case["form"] == "step":
        s["dlogits"] = torch.empty_like(x)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return _plain_scores(state, case) if case["op"] == "scores" else _plain_distill(state, case)


def _run_own(s, case):
    import byte_level_bpe_amd as B
    if case["op"] == "scores":
        t = B.token_logprobs(s["logits"], s["ids"], top_k=min(case["k"], case["vocab"]), scale=s["scale"])
        if case["form"] == "gradient":
            d = B.token_logprobs_backward(s["logits"], s["ids"], t, grad_logprobs=s["g_logprobs"], grad_entropy=s["g_entropy"], scale=s["scale"])
            return {"logprobs": t.logprobs, "entropy": t.entropy, "dlogits": d}
        got = {"logprobs": t.logprobs, "entropy": t.entropy, "lse": t.lse, "ranks": t.ranks}
        return got | {"top_ids": t.top_ids, "top_logprobs": t.top_logprobs} if case["k"] else got
    how = dict(tail=case["tail"], scale=s["scale"])
    if case["form"] == "step":
        t = B.distill_loss(s["logits"], s["top_ids"], s["top"], weights=s["weights"], dlogits=s["dlogits"], **how)
        return {"loss": t.loss, "dlogits": s["dlogits"]}
    t = B.distill_loss(s["logits"], s["top_ids"], s["top"], **how)
    if case["form"] == "loss":
        return {"loss": t.loss}
    return {"loss": t.loss, "dlogits": B.distill_loss_backward(s["weights"], s["logits"], s["top_ids"], s["top"], t, **how)}


def _softmax_parts(z):
    """(z less the row's maximum, its exp, their sum, its log); a row that is minus infinity throughout sums to 0."""
    top = z.amax(1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    d = z - top
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    return top, d, e, total, torch.log(total)


def _plain_scores(s, case):
    x, ids, v = s["logits"], s["ids"].long()[:, None], case["vocab"]
    top, d, e, total, log_total = _softmax_parts(x.float() * s["scale"])
    some, given = total > 0, ids >= 0
    logprob = lambda at: torch.where(some, d.gather(1, at) - log_total, -math.inf)  # noqa: E731
    own_lp = torch.where(given, logprob(ids.clamp(min=0)), 0)
    bounded = d.clamp(min=-1e4)  # 0 * -inf is 0 here
    entropy = torch.where(some, log_total - (e * bounded).sum(1, keepdim=True) / total, 0)
    if case["form"] == "gradient":
        p = torch.where(some, e / total, 0)
        del e
        g, gh = torch.where(given, s["g_logprobs"][:, None], 0), s["g_entropy"][:, None]
        dz = -p * (g + gh * (bounded - log_total + entropy))
        dz.scatter_add_(1, ids.clamp(min=0), g)
        return {"logprobs": own_lp[:, 0], "entropy": entropy[:, 0], "dlogits": (dz * s["scale"]).to(x.dtype)}
    lse = top + log_total
    del e, bounded
    at, j = x.gather(1, ids.clamp(min=0)), torch.arange(v, device=x.device)[None, :]
    before = (x > at) | ((x == at) & (j < ids))
    ranks = torch.where(given[:, 0], before.sum(1) + 1, 0).to(torch.int32)
    got = {"logprobs": own_lp[:, 0], "entropy": entropy[:, 0], "lse": lse[:, 0], "ranks": ranks}
    if case["k"]:
        # values in order as whole numbers, the lower index first among equals
        b = (x.float() + 0.0).view(torch.int32)
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * 2**32 + (2**32 - 1 - j)
        first = torch.topk(key, min(case["k"], v), dim=1).values
        at = 2**32 - 1 - (first & (2**32 - 1))
        got |= {"top_ids": at.to(torch.int32), "top_logprobs": logprob(at)}
    return got


def _plain_distill(s, case):
    x, n, v = s["logits"], case["rows"], case["vocab"]
    ids, lp = s["top_ids"].long(), s["top"].double()
    held = ids >= 0
    lp = lp.masked_fill(~held, -math.inf)
    c = torch.zeros_like(lp[:, :1]) if case["tail"] else torch.logsumexp(lp, 1, keepdim=True)
    q = torch.exp(lp - c.masked_fill(c == -math.inf, 0))
    mass = q.sum(1, keepdim=True)
    rest = (1 - mass).clamp(min=0) if case["tail"] else torch.zeros_like(mass)
    # the student's exponentials in 32 bits, their sums and a row's few numbers in 64: they are differences of near ones
    _, d, e, _, _ = _softmax_parts(x.float() * s["scale"])
    at = ids.clamp(min=0)
    if case["tail"]:
        listed_ = torch.zeros(n, v + 1, dtype=torch.bool, device=x.device).scatter_(1, torch.where(held, ids, v), True)[:, :v]
        high, _, _, other, _ = _softmax_parts(d.masked_fill(listed_, -math.inf))
        named = torch.exp(d.gather(1, at).double() - high.double()).masked_fill(~held, 0).sum(1, keepdim=True)
        log_rest = -torch.log1p(named / other.double())
        log_total = high.double() + torch.log(other.double() + named)
    else:
        log_total = torch.log(e.sum(1, keepdim=True, dtype=torch.float64))
    log_p = d.gather(1, at).double() - log_total
    loss = torch.where(q > 0, q * (torch.log(q.masked_fill(q == 0, 1)) - log_p), 0).sum(1, keepdim=True)
    if case["tail"]:
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest.masked_fill(rest == 0, 1)) - log_rest), 0)
    if case["form"] == "loss":
        return {"loss": loss[:, 0].float()}
    weight = (mass + rest).float()
    p = e.mul_(torch.exp(-log_total).float())
    if case["tail"]:
        share = torch.where(rest > 0, rest * torch.exp(-log_rest), 0).float()
        dz = p * torch.where(listed_, weight, weight - share)
    else:
        dz = p.mul_(weight)
    dz.scatter_add_(1, ids.clamp(min=0), -torch.where(held, q, 0).float())
    return {"loss": loss[:, 0].float(), "dlogits": (dz * (s["weights"][:, None] * s["scale"])).to(x.dtype)}


# ---------------------------------------------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    n, v, size = case["rows"], case["vocab"], 4 if case["dtype"] == "f32" else 2
    grad, k = case["form"] in ("gradient", "step"), case["k"]
    if case["op"] == "scores":
        row = 4 + 8 + (8 if grad else 8 + 8 * k)
        ops = 9 if not grad else 16
    else:
        row = 8 * k + 4 + (4 if grad else 0)
        ops = 4 if not grad else 7
    return {"bytes": n * v * size * (2 if grad else 1) + n * row, "flops": ops * n * v}


def _row_blocks(case):
    step = max(1, 2**27 // case["vocab"])
    return [slice(a, min(case["rows"], a + step)) for a in range(0, case["rows"], step)]


def exact(case, seed):
    s = prepare(case, seed)
    parts = [(_exact_scores if case["op"] == "scores" else _exact_distill)(s, case, rows) for rows in _row_blocks(case)]
    return {name: None if parts[0][name] is None else torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_scores(s, case, rows):
    """The definition: log_softmax, and its own derivative for the gradient."""
    x = s["logits"][rows].double().requires_grad_(case["form"] == "gradient")
    ids = s["ids"][rows].long()
    logp = torch.log_softmax(x * s["scale"], dim=1)
    lp = logp[torch.arange(len(ids), device=x.device), ids.clamp(min=0)].masked_fill(ids < 0, 0)
    logp0 = logp.masked_fill(logp == -math.inf, 0)
    entropy = -(torch.exp(logp) * logp0).sum(1)
    got = {"logprobs": lp.detach(), "entropy": entropy.detach()}
    if case["form"] == "gradient":
        (got["dlogits"],) = torch.autograd.grad((lp, entropy), x, (s["g_logprobs"][rows].double(), s["g_entropy"][rows].double()))
        return got
    got |= {"lse": torch.logsumexp(x * s["scale"], 1), "ranks": None}
    if case["k"]:  # (equal values are equal log probabilities, whichever comes first)
        got |= {"top_ids": None, "top_logprobs": torch.topk(logp, min(case["k"], case["vocab"]), dim=1).values}
    return got


def _exact_distill(s, case, rows):
    x = s["logits"][rows].double().requires_grad_(case["form"] != "loss")
    ids, lp = s["top_ids"][rows].long(), s["top"][rows].double()
    held = ids >= 0
    logp = torch.log_softmax(x * s["scale"], dim=1)
    q = torch.exp(lp).masked_fill(~held, 0)
    mass = q.sum(1, keepdim=True)
    if not case["tail"]:
        q = q / mass.masked_fill(mass == 0, 1)
    kl = lambda a, log_b: torch.where(a > 0, torch.xlogy(a, a) - a * log_b, 0)  # noqa: E731
    loss = kl(q, logp.gather(1, ids.clamp(min=0))).sum(1)
    if case["tail"]:
        listed_ = torch.zeros(x.shape[0], x.shape[1] + 1, dtype=torch.bool, device=x.device).scatter_(1, torch.where(held, ids, x.shape[1]), True)[:, :-1]
        loss = loss + kl((1 - mass[:, 0]).clamp(min=0), torch.logsumexp(logp.masked_fill(listed_, -math.inf), 1))
    got = {"loss": loss.detach()}
    if case["form"] != "loss":
        (got["dlogits"],) = torch.autograd.grad(loss, x, s["weights"][rows].double())
    return got
