"""From logits to ids: scores of given tokens (log probability, entropy, rank,
the most likely alternatives) and distillation from a teacher's alternatives,
each with its gradient.

Argument marshalling and the recording of gradients only, as in serving.py, and
in its manner: calls enqueue on the current stream (or the one given) and return
without synchronising; given their outputs they allocate nothing, so they can be
captured into a HIP graph.

    ids, id_off, n = tok.encode_device(text, seg_off, allow, total)
    scored = token_logprobs(teacher_logits, next_ids, top_k=64)
    loss = distill_loss(student_logits, scored.top_ids, scored.top_logprobs, tail=True).loss
    loss.mean().backward()
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple

import torch

from . import _load
from .serving import _DTYPES, _On, _bad, _check, _dense, _no_tangents, _short, _wants_grad, _written_to

_fns = None


def _lib():
    global _fns
    if _fns is None:
        lib = _load()
        P, U32, U64, I64, I, F = (C.c_void_p, C.c_uint32, C.c_uint64, C.c_int64, C.c_int, C.c_float)
        X = [I, P, I64, U64, U32]  # dtype, logits, row stride, rows, vocabulary
        for name, args in {
            "bbpe_token_logprobs_workspace_bytes": [I, U64, U32, U32, C.POINTER(U64)],
            "bbpe_token_logprobs": X + [P, U32, F] + 8 * [P] + [U64, P],
            "bbpe_token_logprobs_backward": X + [P, U32, F] + 8 * [P] + [I64, P],
            "bbpe_distill_loss_workspace_bytes": [I, U64, U32, C.POINTER(U64)],
            "bbpe_distill_loss": X + [P, P, U32, I, F] + 5 * [P] + [I64, P, U64, P],
            "bbpe_distill_loss_backward": X + [P, P, U32, I, F] + 3 * [P] + [I64, P],
        }.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = I, args
        _fns = lib
    return _fns


def _logits(what, t):
    """[rows, vocabulary] with contiguous rows: the C call's first arguments."""
    if t.dim() != 2 or t.dtype not in _DTYPES or (t.stride(1) != 1 and t.shape[1] > 1):
        _bad("%s: logits [rows, vocabulary] of bfloat16, float16 or float32 with contiguous rows are wanted, got %s %s strides %s"
             % (what, t.dtype, list(t.shape), t.stride()))
    return _DTYPES[t.dtype], t.data_ptr(), t.stride(0), t.shape[0], t.shape[1]


def _gradient(what, t, logits):
    """The gradient's tensor: pointer and row stride."""
    if t.dtype is not logits.dtype or t.device != logits.device or t.shape != logits.shape or (t.stride(1) != 1 and t.shape[1] > 1):
        _bad("%s: dlogits: a %s tensor of shape %s with contiguous rows on %s is wanted, got %s %s strides %s on %s" %
             (what, logits.dtype, list(logits.shape), logits.device, t.dtype, list(t.shape), t.stride(), t.device))
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        _bad("%s: dlogits: rows share memory: strides %s" % (what, t.stride()))
    return t.data_ptr(), t.stride(0)


def _room(size_of, given, dev, what, *args):
    """The workspace: (tensor or None, pointer, bytes).  size_of: the library's function that tells its size."""
    if given is None:
        size = C.c_uint64()
        _check(size_of(*args, C.byref(size)), what)
        if size.value == 0:
            return None, None, 0
        given = torch.empty(size.value, dtype=torch.uint8, device=dev)
    return given, _dense("workspace", given, torch.uint8, (None,), dev), given.numel()


def _or_none(name, t, shape, dev):
    return None if t is None else _dense(name, t, torch.float32, shape, dev)


# ---- scores ----
class TokenLogprobs(NamedTuple):
    """What token_logprobs returns, a row each."""
    logprobs: torch.Tensor      # float32 [n]
    entropy: torch.Tensor       # float32 [n]
    lse: torch.Tensor           # float32 [n]
    ranks: torch.Tensor         # int32 [n], from 1
    top_ids: torch.Tensor       # int32 [n, top_k]
    top_logprobs: torch.Tensor  # float32 [n, top_k]
    stats: torch.Tensor         # float32 [n, 2], for the gradient


class _TokenLogprobs(torch.autograd.Function):
    """token_logprobs where gradients are wanted (its forward runs without grad mode, so plainly)."""

    @staticmethod
    def forward(ctx, logits, ids, top_k, scale):
        got = token_logprobs(logits, ids, top_k, scale)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(got.ranks, got.top_ids, got.stats)
        ctx.save_for_backward(logits, ids, got.entropy, got.top_ids, got.stats)
        ctx.scale = scale
        return tuple(got)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logprobs, g_entropy, g_lse, _ranks, _ids, g_top, _stats):
        logits, ids, entropy, top_ids, stats = ctx.saved_tensors
        scored = TokenLogprobs(None, entropy, None, None, top_ids, None, stats)
        # (a sum's gradient, for one, is broadcast)
        grads = [g if g is None else g.contiguous() for g in (g_logprobs, g_entropy, g_lse, g_top)]
        return token_logprobs_backward(logits, ids, scored, *grads, scale=ctx.scale), None, None, None


def token_logprobs(logits, ids, top_k: int = 0, scale: float = 1.0, out=None, workspace=None, stream=None) -> TokenLogprobs:
    """Scores of the tokens ids [n] under softmax(scale * logits [n,
    vocabulary]) (bbpe_token_logprobs).

    logits: bfloat16, float16 or float32, contiguous rows at any stride; ids:
    int32, below 0 where a row has no token; top_k: alternatives a row, up to
    256, in the order of logits, the lower id first among equals; scale: 1 /
    temperature; out: a TokenLogprobs to write into; workspace: uint8, for few
    rows (bbpe_token_logprobs_workspace_bytes).

    Where grad mode is on and logits require grad, logprobs, entropy, lse and
    top_logprobs carry their gradients (once, backward: inputs with tangents are
    refused); into given outputs there are none, and such a call is refused."""
    if out is None and workspace is None and stream is None:
        got = _short.token_logprobs(logits, ids, top_k, scale)
        if got is not NotImplemented:
            return tuple.__new__(TokenLogprobs, got)
    _no_tangents("token_logprobs", logits)
    if _wants_grad(logits):
        if out is not None or workspace is not None:
            _bad("token_logprobs: no gradients into given outputs or workspaces; call it under torch.no_grad()")
        with _On(logits.device, stream, "token_logprobs") as on:
            got = TokenLogprobs(*_TokenLogprobs.apply(logits, ids, top_k, scale))
            on.keep(logits, ids)
        return got
    dev = logits.device
    with _On(dev, stream, "token_logprobs") as on:
        x = _logits("token_logprobs", logits)
        n, f32, i32 = logits.shape[0], torch.float32, torch.int32
        if not 0 <= top_k <= min(256, logits.shape[1]):  # (before anything is allocated)
            _bad("token_logprobs: top_k %d of a vocabulary of %d" % (top_k, logits.shape[1]))
        given = out or ()
        if out is None:
            shapes = ((n,), f32), ((n,), f32), ((n,), f32), ((n,), i32), ((n, top_k), i32), ((n, top_k), f32), ((n, 2), f32)
            out = TokenLogprobs(*(torch.empty(s, dtype=t, device=dev) for s, t in shapes))
        room, *space = _room(_lib().bbpe_token_logprobs_workspace_bytes, workspace, dev, "token_logprobs", x[0], n, x[4], top_k)
        st = _lib().bbpe_token_logprobs(
            *x, _dense("ids", ids, i32, (n,), dev), top_k, float(scale), *(
                _dense(name, t, f32, (n,), dev) for name, t in (("logprobs", out.logprobs), ("entropy", out.entropy), ("lse", out.lse))),
            _dense("ranks", out.ranks, i32, (n,), dev), _dense("top_ids", out.top_ids, i32, (n, top_k), dev),
            _dense("top_logprobs", out.top_logprobs, f32, (n, top_k), dev), _dense("stats", out.stats, f32, (n, 2), dev), *space, on.handle)
        _check(st, "token_logprobs")
        _written_to(*given)
        on.keep(logits, ids, room, *out)
    return out


def token_logprobs_backward(logits, ids, scored: TokenLogprobs, grad_logprobs=None, grad_entropy=None, grad_lse=None,
                            grad_top=None, scale: float = 1.0, dlogits=None, stream=None):
    """The gradient of the logits from those of token_logprobs' outputs
    (bbpe_token_logprobs_backward): float32 [n], grad_top [n, top_k], None for
    zeros.  scored: what token_logprobs returned for these logits, ids and
    scale.  dlogits may be logits.  It carries no gradient of its own."""
    if dlogits is None and stream is None:
        got = _short.token_logprobs_backward(logits, ids, scored.entropy, scored.top_ids, scored.stats, grad_logprobs, grad_entropy,
                                             grad_lse, grad_top, scale)
        if got is not NotImplemented:
            return got
    _no_tangents("token_logprobs_backward", logits, scored.entropy, grad_logprobs, grad_entropy, grad_lse, grad_top)
    dev = logits.device
    with _On(dev, stream, "token_logprobs_backward") as on:
        x = _logits("token_logprobs_backward", logits)
        n, f32, i32, k = logits.shape[0], torch.float32, torch.int32, scored.top_ids.shape[-1]
        given = dlogits
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        st = _lib().bbpe_token_logprobs_backward(
            *x, _dense("ids", ids, i32, (n,), dev), k, float(scale), _dense("entropy", scored.entropy, f32, (n,), dev),
            _dense("top_ids", scored.top_ids, i32, (n, k), dev), _dense("stats", scored.stats, f32, (n, 2), dev),
            _or_none("grad_logprobs", grad_logprobs, (n,), dev), _or_none("grad_entropy", grad_entropy, (n,), dev),
            _or_none("grad_lse", grad_lse, (n,), dev), _or_none("grad_top", grad_top, (n, k), dev),
            *_gradient("token_logprobs_backward", dlogits, logits), on.handle)
        _check(st, "token_logprobs_backward")
        _written_to(given)
        on.keep(logits, ids, scored.entropy, scored.top_ids, scored.stats, grad_logprobs, grad_entropy, grad_lse, grad_top, dlogits)
    return dlogits


# ---- distillation ----
class DistillLoss(NamedTuple):
    """What distill_loss returns, a row each."""
    loss: torch.Tensor   # float32 [n]
    lse: torch.Tensor    # float32 [n], the student's
    stats: torch.Tensor  # float32 [n, 4], for the gradient


class _DistillLoss(torch.autograd.Function):
    """distill_loss where gradients are wanted (its forward runs without grad mode, so plainly)."""

    @staticmethod
    def forward(ctx, logits, top_ids, top_logprobs, tail, scale):
        got = distill_loss(logits, top_ids, top_logprobs, tail, scale)
        ctx.mark_non_differentiable(got.lse, got.stats)
        ctx.save_for_backward(logits, top_ids, top_logprobs, got.stats)
        ctx.how = tail, scale
        return tuple(got)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _lse, _stats):
        *args, stats = ctx.saved_tensors
        return distill_loss_backward(grad.contiguous(), *args, DistillLoss(None, None, stats), *ctx.how), None, None, None, None


def _lists(what, top_ids, top_logprobs, n, dev):
    k = top_ids.shape[1] if top_ids.dim() == 2 else -1
    return (_dense(what + ": top_ids", top_ids, torch.int32, (n, k), dev),
            _dense(what + ": top_logprobs", top_logprobs, torch.float32, (n, k), dev), k)


def distill_loss(logits, top_ids, top_logprobs, tail: bool = False, scale: float = 1.0, weights=None, dlogits=None, out=None,
                 workspace=None, stream=None) -> DistillLoss:
    """Divergence of softmax(scale * logits [n, vocabulary]) from a teacher's
    listed tokens, top_ids (int32) and top_logprobs (float32) [n, k], k up to
    256 (bbpe_distill_loss).

    top_logprobs are the teacher's log probabilities at the same temperature
    (token_logprobs' with this scale).  tail False: the list made to sum to 1
    against the student's whole distribution; True: what the list leaves of 1
    against the student's sum over tokens not listed (where those are masked by
    minus infinity, what rounding leaves is none; under a finite mask it counts,
    times what the mask takes off).  Entries with ids outside the vocabulary are
    not there: -1 fills up a shorter list; a row with none has loss 0 and no
    gradient.

    workspace: uint8, for few rows (bbpe_distill_loss_workspace_bytes).

    With weights (float32 [n]) and dlogits (which may be logits) the call also
    writes the gradient of (weights * loss).sum(): one call of a training step
    that knows its weights.  Otherwise, where grad mode is on and logits
    require grad, loss carries its gradient (once, backward: inputs with tangents
    are refused; the teacher has none)."""
    if (weights is None) != (dlogits is None):
        _bad("distill_loss: weights and dlogits are given together or not at all")
    if out is None and workspace is None and stream is None:
        got = _short.distill_loss(logits, top_ids, top_logprobs, tail, scale, weights, dlogits)
        if got is not NotImplemented:
            return tuple.__new__(DistillLoss, got)
    _no_tangents("distill_loss", logits, top_logprobs, weights)
    if _wants_grad(logits, top_logprobs, weights):
        if out is not None or workspace is not None or dlogits is not None or top_logprobs.requires_grad:
            _bad("distill_loss: no gradients into given outputs or workspaces, nor of the teacher or the weights; call it under torch.no_grad()")
        with _On(logits.device, stream, "distill_loss") as on:
            got = DistillLoss(*_DistillLoss.apply(logits, top_ids, top_logprobs, tail, scale))
            on.keep(logits, top_ids, top_logprobs)
        return got
    dev = logits.device
    with _On(dev, stream, "distill_loss") as on:
        x = _logits("distill_loss", logits)
        n, f32 = logits.shape[0], torch.float32
        ids, lp, k = _lists("distill_loss", top_ids, top_logprobs, n, dev)
        given = (dlogits, *(out or ()))
        if out is None:
            out = DistillLoss(*(torch.empty(s, dtype=f32, device=dev) for s in ((n,), (n,), (n, 4))))
        room, *space = _room(_lib().bbpe_distill_loss_workspace_bytes, workspace, dev, "distill_loss", x[0], n, x[4])
        st = _lib().bbpe_distill_loss(
            *x, ids, lp, k, bool(tail), float(scale), _dense("loss", out.loss, f32, (n,), dev), _dense("lse", out.lse, f32, (n,), dev),
            _dense("stats", out.stats, f32, (n, 4), dev), _or_none("weights", weights, (n,), dev),
            *((None, 0) if dlogits is None else _gradient("distill_loss", dlogits, logits)), *space, on.handle)
        _check(st, "distill_loss")
        _written_to(*given)
        on.keep(logits, top_ids, top_logprobs, weights, dlogits, room, *out)
    return out


def distill_loss_backward(grad_loss, logits, top_ids, top_logprobs, distilled: DistillLoss, tail: bool = False, scale: float = 1.0,
                          dlogits=None, stream=None):
    """The gradient of the logits from that of distill_loss' loss, float32 [n]
    (bbpe_distill_loss_backward).  distilled: what distill_loss returned for
    these arguments.  dlogits may be logits.  It carries no gradient of its own."""
    if dlogits is None and stream is None:
        got = _short.distill_loss_backward(grad_loss, logits, top_ids, top_logprobs, distilled.stats, tail, scale)
        if got is not NotImplemented:
            return got
    _no_tangents("distill_loss_backward", grad_loss, logits, top_logprobs)
    dev = logits.device
    with _On(dev, stream, "distill_loss_backward") as on:
        x = _logits("distill_loss_backward", logits)
        n, f32 = logits.shape[0], torch.float32
        ids, lp, k = _lists("distill_loss_backward", top_ids, top_logprobs, n, dev)
        given = dlogits
        if dlogits is None:
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        st = _lib().bbpe_distill_loss_backward(
            *x, ids, lp, k, bool(tail), float(scale), _dense("stats", distilled.stats, f32, (n, 4), dev),
            _dense("grad_loss", grad_loss, f32, (n,), dev), *_gradient("distill_loss_backward", dlogits, logits), on.handle)
        _check(st, "distill_loss_backward")
        _written_to(given)
        on.keep(logits, top_ids, top_logprobs, distilled.stats, grad_loss, dlogits)
    return dlogits
