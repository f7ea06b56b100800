"""From ids to attention: block tables and slot maps from request lengths, the
norm of queries and keys with their rotation, and attention of new tokens (a
tree of drafts, a chain, one token) over a paged cache.

Argument marshalling only, as in the package's encode calls, and the recording
of qk_norm_rope's gradient: the work is in the HIP kernels behind
include/bbpe.h.  Every call enqueues on the current stream (or the one given)
and returns without synchronising; given buffers (`out=` and the like, and a
workspace) it allocates nothing, so it can be captured into a HIP graph.

    ids, id_off, n = tok.encode_device(text, seg_off, allow, total)
    plan = block_tables(id_off, ctx_len, free_pages, table, 64, n)
    q, _ = qk_norm_rope(q, k, w_q, w_k, plan.positions, inv_freq,
                        v=v, cache=cache, slots=plan.slots)
    out = tree_attention(q, cache, table, id_off, ctx_len)
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import os
from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from . import BBPEError, E_INVALID_ARG, HERE, _load

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # BBPE_BF16, BBPE_F16, BBPE_F32


class _CacheStruct(C.Structure):
    """bbpe_paged_cache"""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("n_pages", C.c_uint64),
                ("page_size", C.c_uint32), ("n_kv_heads", C.c_uint32), ("head_dim", C.c_uint32),
                ("dtype", C.c_int32), ("page_stride", C.c_int64), ("head_stride", C.c_int64),
                ("token_stride", C.c_int64)]


_fns = None


def _lib():
    global _fns
    if _fns is None:
        lib = _load()
        P, U32, U64, I64, I, F = (C.c_void_p, C.c_uint32, C.c_uint64, C.c_int64, C.c_int, C.c_float)
        R = [P, I64, I64]  # rows: pointer, token stride, head stride
        O = C.POINTER(U64)
        for name, args in {
            "bbpe_block_tables_workspace_bytes": [U32, O],
            "bbpe_block_tables": [P, P, U32, P, U64, P, U64, U32, U32, U64, P, P, P, P, P, P, P, U64, P],
            "bbpe_qk_norm_rope": [I, U64, U32, U32, U32, U32, I, F] + 3 * R + [P, P, P, P] + 2 * R + [P, P, P],
            "bbpe_qk_norm_rope_backward_workspace_bytes": [U64, U32, O],
            "bbpe_qk_norm_rope_backward":
                [I, U64, U32, U32, U32, U32, I, F] + 4 * R + [P, P, P, P] + 2 * R + [P, P, P, U64, P],
            "bbpe_tree_attention_workspace_bytes": [U64, U32, U32, P, O],
            "bbpe_tree_attention": R + [U64, U32, P, P, U64, U32, P, P, U32, P, U32, F] + R + [P, P, U64, P],
        }.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = I, args
        _fns = lib
    return _fns


def _short_way():
    """The _serving extension (csrc/bbpe_torch.cpp), which takes plain calls in
    one step and leaves the others, by NotImplemented, to the code here."""
    path = os.path.join(HERE, "_serving.so")
    if not os.path.exists(path):
        raise ImportError("_serving.so is not built; run python -m byte_level_bpe_amd.build")
    spec = importlib.util.spec_from_file_location(__package__ + "._serving", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    lib = _lib()
    mod.bind(*(C.cast(getattr(lib, "bbpe_" + n), C.c_void_p).value for n in (
        "block_tables", "qk_norm_rope", "qk_norm_rope_backward_workspace_bytes", "qk_norm_rope_backward",
        "tree_attention_workspace_bytes", "tree_attention", "token_logprobs_workspace_bytes", "token_logprobs",
        "token_logprobs_backward", "distill_loss_workspace_bytes", "distill_loss", "distill_loss_backward")))
    return mod


_short = _short_way()


def _bad(what: str):
    err = BBPEError(E_INVALID_ARG, what)
    raise err


def _check(st: int, what: str):
    if st:
        raise BBPEError(st, what)


def _dense(name, t, dtype, shape, dev):
    """A contiguous tensor of this type and shape (None: any length), on dev."""
    if t.dtype is not dtype or t.device != dev or len(t.shape) != len(shape) or not t.is_contiguous() or \
            any(w is not None and w != n for w, n in zip(shape, t.shape)):
        _bad("%s: a contiguous %s tensor of shape %s on %s is wanted, got %s %s on %s" %
             (name, dtype, list(shape), dev, t.dtype, list(t.shape), t.device))
    return t.data_ptr()


def _rows(name, t, dtype, shape, dev):
    """[tokens, heads, dim] with a contiguous last dimension: pointer, token and head strides."""
    if t.dtype is not dtype or t.device != dev or t.shape != shape or (t.stride(2) != 1 and shape[2] > 1):
        _bad("%s: a %s tensor of shape %s, contiguous in its last dimension, on %s is wanted, got %s %s strides %s on %s"
             % (name, dtype, list(shape), dev, t.dtype, list(t.shape), t.stride(), t.device))
    return t.data_ptr(), t.stride(0), t.stride(1)


def _written(name, t, dtype, shape, dev):
    """_rows of a tensor to be written, whose rows must be places of their own."""
    rows = _rows(name, t, dtype, shape, dev)
    if any(t.stride(d) == 0 and shape[d] > 1 for d in (0, 1)):
        _bad("%s: rows share memory: strides %s" % (name, t.stride()))
    return rows


_NONE = (None, 0, 0)


class _On:
    """The device and stream of a call: makes them current where they are not,
    so that what the call allocates belongs to its stream, and keeps tensors of
    other streams alive until the stream is past the call."""

    def __init__(self, dev, stream, what):
        if dev.type != "cuda":
            _bad("%s: tensors on a GPU are wanted, got %s" % (what, dev))
        self.ctx = None
        here = torch.cuda.current_device()
        if stream is not None:
            if stream.device != dev:
                _bad("%s: the stream is on %s, the tensors on %s" % (what, stream.device, dev))
            if dev.index != here or stream != torch.cuda.current_stream():
                self.ctx = torch.cuda.stream(stream)
        elif dev.index != here:
            self.ctx = torch.cuda.device(dev)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        self.stream = torch.cuda.current_stream()
        self.handle = self.stream.cuda_stream
        return self

    def keep(self, *tensors):
        if self.ctx is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


# ---- block tables ----
class BlockTables(NamedTuple):
    """What block_tables wrote besides the table."""
    slots: torch.Tensor      # int64 [n_tokens]
    positions: torch.Tensor  # int32 [n_tokens]
    requests: torch.Tensor   # int32 [n_tokens]
    seq_len: torch.Tensor    # int32 [n_req]
    status: torch.Tensor     # int64 [4]: code, first failed request, pages taken, tokens placed

    def wait(self):
        """Reads the status back (this synchronises): (pages taken, tokens
        placed), or raises with the first failed request's error (.request)."""
        code, request, pages, tokens = self.status.tolist()
        if code:
            err = BBPEError(code, "block_tables: request %d" % request)
            err.request = request
            raise err
        return pages, tokens


def block_tables(q_off, ctx_len, free_pages, table, page_size: int, n_tokens: int, depth=None, out=None,
                 workspace=None, stream=None) -> BlockTables:
    """Pages, slots and positions for the new tokens of every request
    (bbpe_block_tables).

    q_off: int64 [n_req + 1], an encode call's id_off; ctx_len: int32 [n_req]
    tokens already cached; free_pages: int32, handed out in order; table: int32
    [n_req, width], updated in place (rows may be strided); n_tokens: length of
    the per-token outputs; depth: int32 [n_tokens], a drafted token's depth in
    its tree; out: a BlockTables to write into; workspace: uint8, for more than
    4,096 requests."""
    if out is None and workspace is None and stream is None:
        got = _short.block_tables(q_off, ctx_len, free_pages, table, page_size, n_tokens, depth)
        if got is not NotImplemented:
            return tuple.__new__(BlockTables, got)
    dev = q_off.device
    n = ctx_len.shape[0] if ctx_len.dim() == 1 else -1
    with _On(dev, stream, "block_tables") as on:
        if table.dtype is not torch.int32 or table.device != dev or table.dim() != 2 or table.shape[0] != n or \
                (table.stride(1) != 1 and table.shape[1] > 1) or table.stride(0) < 0:
            _bad("block_tables: table: an int32 tensor [%d, width] with contiguous rows on %s is wanted, got %s %s on %s" %
                 (n, dev, table.dtype, list(table.shape), table.device))
        n_tokens = int(n_tokens)
        if not 0 <= n_tokens < 1 << 31 or not 0 < page_size <= 1 << 30:  # (before anything is allocated)
            _bad("block_tables: n_tokens %d, page_size %d" % (n_tokens, page_size))
        if out is None:
            up = (n_tokens + 3) // 4 * 4
            i32 = torch.empty(up + n_tokens, dtype=torch.int32, device=dev)
            out = BlockTables(torch.empty(n_tokens, dtype=torch.int64, device=dev), i32[:n_tokens], i32[up:],
                              torch.empty(n, dtype=torch.int32, device=dev), torch.empty(4, dtype=torch.int64, device=dev))
        lib, need = _lib(), 0
        if n > 4096:
            size = C.c_uint64()
            _check(lib.bbpe_block_tables_workspace_bytes(n, C.byref(size)), "block_tables")
            need = size.value
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        i64, i32 = torch.int64, torch.int32
        st = lib.bbpe_block_tables(
            _dense("q_off", q_off, i64, (n + 1,), dev), _dense("ctx_len", ctx_len, i32, (n,), dev), n,
            _dense("free_pages", free_pages, i32, (None,), dev), free_pages.shape[0],
            table.data_ptr(), table.stride(0), table.shape[1], page_size, n_tokens,
            None if depth is None else _dense("depth", depth, i32, (n_tokens,), dev),
            _dense("slots", out.slots, i64, (n_tokens,), dev),
            _dense("positions", out.positions, i32, (n_tokens,), dev),
            _dense("requests", out.requests, i32, (n_tokens,), dev),
            _dense("seq_len", out.seq_len, i32, (n,), dev), _dense("status", out.status, i64, (4,), dev),
            None if workspace is None else _dense("workspace", workspace, torch.uint8, (None,), dev),
            0 if workspace is None else workspace.numel(), on.handle)
        _check(st, "block_tables")
        on.keep(q_off, ctx_len, free_pages, table, depth, workspace, *out)
    return out


# ---- the paged cache ----
class PagedCache:
    """A paged key/value cache over two tensors [n_pages, n_kv_heads,
    page_size, head_dim] of the same type (bfloat16 or float16), shape and
    strides, contiguous in the last dimension.  Views of one allocation will do,
    as will another order of heads and tokens in memory.  It is a handle to
    their memory: other tensors want another PagedCache."""

    def __setattr__(self, name, value):
        # the kernels' description of the cache is made once, from these
        if "_p" in self.__dict__ and name in self.__dict__:
            raise AttributeError("PagedCache: %s is fixed; make another PagedCache" % name)
        super().__setattr__(name, value)

    def __init__(self, k, v):
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float16) or k.shape != v.shape or \
                k.stride() != v.stride() or k.dtype is not v.dtype or k.device != v.device or k.stride(3) != 1:
            _bad("PagedCache: two bfloat16 or float16 tensors [pages, heads, page, dim] alike are wanted, got %s %s and %s %s"
                 % (k.dtype, list(k.shape), v.dtype, list(v.shape)))
        if any(s % 8 for s in k.stride()[:3]) or k.data_ptr() % 16 or v.data_ptr() % 16:
            _bad("PagedCache: rows are not 16-byte aligned: strides %s" % (k.stride(),))
        self.k, self.v = k, v
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        self._s = _CacheStruct(k.data_ptr(), v.data_ptr(), self.n_pages, self.page_size, self.n_kv_heads,
                               self.head_dim, _DTYPES[k.dtype], k.stride(0), k.stride(1), k.stride(2))
        self._p = C.addressof(self._s)


# ---- norm and rotation ----
def _norm_args(what, q, k, q_weight, k_weight, positions, inv_freq):
    if q.dim() != 3 or k.dim() != 3 or q.dtype not in _DTYPES:
        _bad("%s: q and k [tokens, heads, dim] of bfloat16, float16 or float32 are wanted, got %s %s, %s %s" %
             (what, q.dtype, list(q.shape), k.dtype, list(k.shape)))
    dev, (n, hq, dim), hk = q.device, q.shape, k.shape[1]
    freq = _dense("inv_freq", inv_freq, torch.float32, (None,), dev)
    ws = [None if w is None else _dense(name, w, q.dtype, (dim,), dev)
          for name, w in (("q_weight", q_weight), ("k_weight", k_weight))]
    return (n, hq, hk, dim, 2 * inv_freq.shape[0], ws,
            _dense("positions", positions, torch.int32, (n,), dev), freq)


def _no_tangents(what, *tensors):
    """Refuses inputs of forward-mode differentiation, whose tangents the kernels would drop."""
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        _bad("%s: no forward-mode gradients, and an input carries a tangent; unpack it, or differentiate backward" % what)


def _written_to(*tensors):
    """Counts the tensors given to write into as changed, as torch does its own: a backward pass that has saved one of
    them raises instead of reading what is there now."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _wants_grad(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class _QkNormRope(torch.autograd.Function):
    """qk_norm_rope where gradients are wanted (its forward runs without grad mode, so plainly)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.how = (eps, interleaved)
        return qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_q, grad_k):
        # (a sum's gradient, for one, is broadcast over the last dimension too)
        grad_q, grad_k = (g if g.stride(2) == 1 else g.contiguous() for g in (grad_q, grad_k))
        weights = ctx.saved_tensors[2:4]
        dq, dk, *dw = qk_norm_rope_backward(grad_q, grad_k, *ctx.saved_tensors, *ctx.how)
        return (dq, dk, *(d if w is None else d.to(w.dtype) for d, w in zip(dw, weights)), None, None, None, None)


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, v=None, cache=None, slots=None, stream=None):
    """RMS norm of every head's row of q [n, n_q_heads, dim] and k [n,
    n_kv_heads, dim], then the rotation of its first 2 * len(inv_freq) elements
    by positions * inv_freq (bbpe_qk_norm_rope).  Returns (q_out, k_out).

    With a PagedCache, v and slots (block_tables'), keys and values go to their
    slots, and k_out is None unless given; the three come together.  Inputs may
    be strided over tokens and heads; q_out may be q and k_out k.  A weight of
    None is ones.

    Where grad mode is on and an input requires grad, the outputs carry the
    gradients of q, k and the weights (once, backward; not those of positions and
    inv_freq).  Into a cache or into given outputs there are none: such a call
    is refused."""
    if not (cache is None) == (v is None) == (slots is None):
        _bad("qk_norm_rope: cache, v and slots are given together or not at all")
    if q_out is None and k_out is None and stream is None:
        got = (_short.qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, None, None, None, None)
               if cache is None else
               _short.qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, v, slots, cache.k,
                                   cache._p))
        if got is not NotImplemented:
            return got
    _no_tangents("qk_norm_rope", q, k, q_weight, k_weight, inv_freq, v)
    if _wants_grad(q, k, q_weight, k_weight, inv_freq, v):
        if cache is not None or q_out is not None or k_out is not None or inv_freq.requires_grad:
            _bad("qk_norm_rope: no gradients into a cache or given outputs, nor of inv_freq; call it under torch.no_grad()")
        with _On(q.device, stream, "qk_norm_rope") as on:
            got = _QkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved)
            on.keep(q, k, q_weight, k_weight, positions, inv_freq)
        return got
    dev, dt = q.device, q.dtype
    with _On(dev, stream, "qk_norm_rope") as on:
        n, hq, hk, dim, rot, ws, pos, freq = _norm_args("qk_norm_rope", q, k, q_weight, k_weight, positions, inv_freq)
        if cache is not None and (cache.device != dev or cache.dtype is not dt):
            _bad("qk_norm_rope: the cache is %s on %s, q %s on %s" % (cache.dtype, cache.device, dt, dev))
        given = q_out, k_out
        if q_out is None:
            q_out = torch.empty((n, hq, dim), dtype=dt, device=dev)
        if k_out is None and cache is None:
            k_out = torch.empty((n, hk, dim), dtype=dt, device=dev)
        kshape = (n, hk, dim)
        st = _lib().bbpe_qk_norm_rope(
            _DTYPES[dt], n, hq, hk, dim, rot, interleaved, eps,
            *_rows("q", q, dt, q.shape, dev), *_rows("k", k, dt, kshape, dev),
            *(_NONE if cache is None else _rows("v", v, dt, kshape, dev)), ws[0], ws[1], pos, freq,
            *_written("q_out", q_out, dt, q.shape, dev),
            *(_NONE if k_out is None else _written("k_out", k_out, dt, kshape, dev)),
            None if cache is None else cache._p,
            None if cache is None else _dense("slots", slots, torch.int64, (n,), dev), on.handle)
        _check(st, "qk_norm_rope")
        _written_to(*given)
        on.keep(q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out, slots)
        if cache is not None:
            on.keep(cache.k, cache.v)
    return q_out, k_out


def qk_norm_rope_backward(grad_q, grad_k, q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope's inputs from those of its outputs
    (bbpe_qk_norm_rope_backward): (dq, dk, dq_weight, dk_weight), the weights'
    in float32, None where the weight is None.  dq may be grad_q, dk grad_k.
    They carry no gradients of their own."""
    if dq is None and dk is None and workspace is None and stream is None:
        got = _short.qk_norm_rope_backward(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved, grad_q, grad_k)
        if got is not NotImplemented:
            return got
    _no_tangents("qk_norm_rope_backward", grad_q, grad_k, q, k, q_weight, k_weight, inv_freq)
    dev, dt = q.device, q.dtype
    with _On(dev, stream, "qk_norm_rope_backward") as on:
        n, hq, hk, dim, rot, ws, pos, freq = _norm_args("qk_norm_rope_backward", q, k, q_weight, k_weight, positions,
                                                        inv_freq)
        given = dq, dk
        if dq is None:
            dq = torch.empty((n, hq, dim), dtype=dt, device=dev)
        if dk is None:
            dk = torch.empty((n, hk, dim), dtype=dt, device=dev)
        dws = [None if w is None else torch.empty(dim, dtype=torch.float32, device=dev) for w in (q_weight, k_weight)]
        lib, size = _lib(), C.c_uint64()
        _check(lib.bbpe_qk_norm_rope_backward_workspace_bytes(n, dim, C.byref(size)), "qk_norm_rope_backward")
        if workspace is None:
            workspace = torch.empty(size.value, dtype=torch.uint8, device=dev)
        kshape = (n, hk, dim)
        st = lib.bbpe_qk_norm_rope_backward(
            _DTYPES[dt], n, hq, hk, dim, rot, interleaved, eps,
            *_rows("grad_q", grad_q, dt, q.shape, dev), *_rows("grad_k", grad_k, dt, kshape, dev),
            *_rows("q", q, dt, q.shape, dev), *_rows("k", k, dt, kshape, dev), ws[0], ws[1], pos, freq,
            *_written("dq", dq, dt, q.shape, dev), *_written("dk", dk, dt, kshape, dev),
            None if dws[0] is None else dws[0].data_ptr(), None if dws[1] is None else dws[1].data_ptr(),
            _dense("workspace", workspace, torch.uint8, (None,), dev), workspace.numel(), on.handle)
        _check(st, "qk_norm_rope_backward")
        _written_to(*given)
        on.keep(grad_q, grad_k, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, workspace, *dws)
    return dq, dk, dws[0], dws[1]


# ---- attention ----
def tree_attention_workspace_bytes(n_tokens: int, n_req: int, n_q_heads: int, cache: PagedCache) -> int:
    size = C.c_uint64()
    _check(_lib().bbpe_tree_attention_workspace_bytes(n_tokens, n_req, n_q_heads, cache._p, C.byref(size)),
           "tree_attention")
    return size.value


def tree_attention(q, cache: PagedCache, table, q_off, ctx_len, tree_mask=None, scale=None, out=None, lse=None,
                   return_lse: bool = False, workspace=None, stream=None):
    """Attention of q [n_tokens, n_q_heads, dim] over the cache, which holds the
    new tokens' keys and values already (bbpe_tree_attention).  Returns out, or
    (out, lse) with return_lse.

    table, q_off, ctx_len: block_tables' arguments (ctx_len: before the new
    tokens); tree_mask: int64 [n_tokens, words], bit j of row i set where token i
    sees new token j of its request; without it, tokens see themselves and those
    before; scale: dim ** -0.5 by default; lse: float32 [n_tokens, n_q_heads].
    It has no gradient: where grad mode is on, inputs that require grad are
    refused."""
    if out is None and lse is None and workspace is None and stream is None:
        got = _short.tree_attention(q, cache.k, cache._p, table, q_off, ctx_len, tree_mask,
                                    cache.head_dim ** -0.5 if scale is None else scale, return_lse)
        if got is not NotImplemented:
            return got if return_lse else got[0]
    _no_tangents("tree_attention", q, cache.k, cache.v)
    if _wants_grad(q, cache.k, cache.v):
        _bad("tree_attention: it has no gradient, and an input requires grad; call it under torch.no_grad()")
    dev, dt = q.device, q.dtype
    with _On(dev, stream, "tree_attention") as on:
        if q.dim() != 3 or dt is not cache.dtype or dev != cache.device or q.shape[2] != cache.head_dim:
            _bad("tree_attention: q [tokens, heads, %d] of %s on %s is wanted, got %s %s on %s" %
                 (cache.head_dim, cache.dtype, cache.device, dt, list(q.shape), dev))
        n, hq, dim = q.shape
        n_req = ctx_len.shape[0] if ctx_len.dim() == 1 else -1
        if table.dtype is not torch.int32 or table.device != dev or table.dim() != 2 or table.shape[0] != n_req or \
                (table.stride(1) != 1 and table.shape[1] > 1) or table.stride(0) < 0:
            _bad("tree_attention: table: an int32 tensor [%d, width] with contiguous rows on %s is wanted, got %s %s on %s"
                 % (n_req, dev, table.dtype, list(table.shape), table.device))
        given = out, lse
        if out is None:
            out = torch.empty((n, hq, dim), dtype=dt, device=dev)
        if lse is None and return_lse:
            lse = torch.empty((n, hq), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(tree_attention_workspace_bytes(n, n_req, hq, cache), dtype=torch.uint8, device=dev)
        st = _lib().bbpe_tree_attention(
            *_rows("q", q, dt, q.shape, dev), n, hq, cache._p, table.data_ptr(), table.stride(0), table.shape[1],
            _dense("q_off", q_off, torch.int64, (n_req + 1,), dev),
            _dense("ctx_len", ctx_len, torch.int32, (n_req,), dev), n_req,
            None if tree_mask is None else _dense("tree_mask", tree_mask, torch.int64, (n, None), dev),
            0 if tree_mask is None else tree_mask.shape[1], dim ** -0.5 if scale is None else scale,
            *_written("out", out, dt, q.shape, dev),
            None if lse is None else _dense("lse", lse, torch.float32, (n, hq), dev),
            _dense("workspace", workspace, torch.uint8, (None,), dev), workspace.numel(), on.handle)
        _check(st, "tree_attention")
        _written_to(*given)
        on.keep(q, table, q_off, ctx_len, tree_mask, out, lse, workspace, cache.k, cache.v)
    return (out, lse) if return_lse else out
