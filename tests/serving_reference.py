"""Plain forms, in 64 bits on the CPU, of the operators between ids and
attention (byte_level_bpe_amd/serving.py), with the error that one rounding to
the output's type and 32-bit arithmetic can make."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tables(q_off, ctx, free, table, page, n_tokens, depth=None):
    """block_tables, request by request: (table, slots, positions, requests, seq_len, status)."""
    q_off, ctx, free = [int(x) for x in q_off], [int(x) for x in ctx], [int(x) for x in free]
    table = np.array(table, dtype=np.int32).copy()
    n, width = table.shape
    slots = np.full(n_tokens, -1, np.int64)
    pos, req = np.zeros(n_tokens, np.int32), np.full(n_tokens, -1, np.int32)
    seq = np.zeros(n, np.int32)
    taken = placed = start = 0
    code, first = 0, -1
    broken = False
    up = lambda x: -(-x // page)  # noqa: E731
    for r in range(n):
        lo, hi, c = q_off[r], q_off[r + 1], ctx[r]
        broken = broken or lo < 0 or hi < lo or hi > n_tokens
        m, held, err = hi - lo, up(max(c, 0)), 0
        need = 0
        if broken or c < 0 or c + m > 2 ** 31 - 1:
            err = -1
        elif up(c + m) > width:
            err = -5
        else:
            need = up(c + m) - held if m else 0
            mine = start
            start += need
            if need and mine + need > len(free):
                err = -5
        end = held
        if err:
            if code == 0:
                code, first = err, r
            seq[r] = max(c, 0)
        else:
            seq[r] = c + m
            end = held + need
            for b in range(held, end):
                table[r, b] = free[mine + b - held]
            taken += need
            placed += m
            for i in range(m):
                p = c + i
                pg = int(table[r, p // page])
                slots[lo + i] = -1 if pg < 0 else pg * page + p % page
                pos[lo + i] = p if depth is None else c + int(depth[lo + i])
                req[lo + i] = r
        table[r, min(end, width):] = -1
    return table, slots, pos, req, seq, np.array([code, first, taken, placed], np.int64)


def _split(y, rot, inter):
    return (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])


def _merge(like, a, b, rot, inter):
    out = like.clone()
    if inter:
        out[..., 0:rot:2], out[..., 1:rot:2] = a, b
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = a, b
    return out


def norm_rope(x, w, positions, inv_freq, eps, inter):
    """(y, bound on |error| of one rounding to x's type after 32-bit arithmetic)."""
    dtype, rot = x.dtype, 2 * inv_freq.numel()
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    ang = positions.double()[:, None, None] * inv_freq.double()
    a, b = _split(n, rot, inter)
    y = _merge(n, a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin(), rot, inter)
    size = _merge(n.abs(), a.abs() + b.abs(), a.abs() + b.abs(), rot, inter)
    # the sum of squares, root, quotient, two products, the turn and its sine: under 32 steps of size
    return y, half_step(dtype) * y.abs() + 32 * U32 * size + torch.finfo(dtype).tiny * half_step(dtype) * 2


def norm_rope_grad(g, x, w, positions, inv_freq, eps, inter):
    """((dx, bound), (dw, bound)): gradients of norm_rope's y with upstream g."""
    dtype, rot = x.dtype, 2 * inv_freq.numel()
    x, g = x.double(), g.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    ang = positions.double()[:, None, None] * inv_freq.double()
    a, b = _split(g, rot, inter)
    dy = _merge(g, a * ang.cos() + b * ang.sin(), b * ang.cos() - a * ang.sin(), rot, inter)
    size = _merge(g.abs(), a.abs() + b.abs(), a.abs() + b.abs(), rot, inter)
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, h = x * rstd, dy * w
    dx = rstd * (h - n * (h * n).mean(-1, keepdim=True))
    mag = rstd * (size * w.abs() + n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True))
    bound = half_step(dtype) * dx.abs() + 64 * U32 * mag + torch.finfo(dtype).tiny * half_step(dtype) * 2
    rows = max(1, x.shape[0] * x.shape[1])
    return (dx, bound), ((dy * n).sum((0, 1)), (rows + 64) * U32 * (size * n.abs()).sum((0, 1)) + 1e-30)


def visible(ctx, m, mask):
    """[m, ctx + m] truth values: who sees whom."""
    see = np.ones((m, ctx + m), bool)
    if mask is None:
        see[:, ctx:] = np.tril(np.ones((m, m), bool))
    else:
        bits = np.unpackbits(np.ascontiguousarray(mask).view(np.uint8).reshape(m, -1), axis=1, bitorder="little").astype(bool)
        new = np.zeros((m, m), bool)
        k = min(m, bits.shape[1])
        new[:, :k] = bits[:, :k]
        see[:, ctx:] = new
    return see


def attention(q, k_cache, v_cache, table, q_off, ctx, mask=None, scale=None):
    """(out, bound, lse, bound): tree_attention, request by request and head by
    head; only visible keys enter any sum."""
    dtype, (n, hq, dim) = q.dtype, q.shape
    pages, hk, page, _ = k_cache.shape
    scale = dim ** -0.5 if scale is None else scale
    out, lse = torch.zeros(n, hq, dim, dtype=torch.float64), torch.full((n, hq), -math.inf, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    h16 = half_step(dtype)
    for r in range(len(ctx)):
        lo, m, c = int(q_off[r]), int(q_off[r + 1] - q_off[r]), int(ctx[r])
        if m == 0:
            continue
        see = visible(c, m, None if mask is None else mask[lo:lo + m].numpy())
        key = np.arange(c + m)
        blk = key // page
        pg = np.where(blk < table.shape[1], table[r].numpy()[np.minimum(blk, table.shape[1] - 1)], -1)
        see &= ((pg >= 0) & (pg < pages))[None, :]
        pg = np.clip(pg, 0, pages - 1)
        k = k_cache[pg, :, key % page].double()  # [keys, hk, dim]
        v = v_cache[pg, :, key % page].double()
        see = torch.from_numpy(see)
        for h in range(hq):
            kh, vh, x = k[:, h // (hq // hk)], v[:, h // (hq // hk)], q[lo:lo + m, h].double()
            for i in range(m):
                at = see[i].nonzero().squeeze(1)
                if not len(at):
                    continue
                kk, vv = kh[at], vh[at]
                s = kk @ x[i] * scale
                lse[lo + i, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - s.max())
                total = p.sum()
                out[lo + i, h] = (p[:, None] * vv).sum(0) / total
                # 32-bit scores move a weight by ds of itself; weights are rounded once to the cache's type
                ds = (dim + 4) * U32 * abs(scale) * (kk.abs() @ x[i].abs()).max()
                steps = (len(at) + 64) * U32
                mass = (p[:, None] * vv.abs()).sum(0) / total
                small = torch.finfo(dtype).tiny * h16 * 2 * vv.abs().sum(0) / total  # weights below the type's range of steps
                o = h16 * out[lo + i, h].abs() + 1.01 * (h16 + 2 * ds + steps) * mass + small
                tol[lo + i, h] = o
                lse_tol[lo + i, h] = 2 * ds + steps + 2 * U32 * lse[lo + i, h].abs()
    return out, tol, lse, lse_tol
