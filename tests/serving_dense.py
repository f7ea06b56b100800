"""tree_attention's definition in 64 bits on the CPU, a request and a key/value
head at a time (tests/serving_reference.py goes row by row and head by head,
which takes too long for many rows), with the error that the kernels' roundings
can make."""
import math

import numpy as np
import torch

from tests.serving_reference import U32, half_step, visible


def attention(q, k_cache, v_cache, table, q_off, ctx, mask=None, scale=None, flushed=1.0):
    """(out, bound, lse, bound).  Offsets must be whole; contexts are clamped at
    0, and keys past a table's row or on pages outside the cache are not seen.
    flushed: what weights too small for the type may be off by, in its smallest steps."""
    dtype, (n, hq, dim) = q.dtype, q.shape
    pages, hk, page, _ = k_cache.shape
    scale, grp, h16 = dim ** -0.5 if scale is None else scale, hq // hk, half_step(q.dtype)
    out, lse = torch.zeros(n, hq, dim, dtype=torch.float64), torch.full((n, hq), -math.inf, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(ctx)):
        lo, m, c = int(q_off[r]), int(q_off[r + 1] - q_off[r]), max(0, int(ctx[r]))
        if m == 0:
            continue
        keys = min(c + m, table.shape[1] * page)
        key = np.arange(keys)
        pg = table[r].numpy()[key // page]
        held = (pg >= 0) & (pg < pages)
        see = torch.from_numpy(visible(c, m, None if mask is None else mask[lo:lo + m].numpy())[:, :keys] & held[None, :])
        pg = np.where(held, pg, 0)
        for h in range(hk):
            k, v = k_cache[pg, h, key % page].double(), v_cache[pg, h, key % page].double()
            odd = ~torch.isfinite(v)
            v0 = v.masked_fill(odd, 0)
            x = q[lo:lo + m, h * grp:(h + 1) * grp].double()  # [m, grp, dim]
            at = see[:, None, :].expand(m, grp, keys)
            s = (x @ k.T * scale).masked_fill(~at, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - top.masked_fill(top == -math.inf, 0))
            total = p.sum(-1, keepdim=True)
            some = total != 0
            over = torch.where(some, total, 1)
            o = p @ v0 / over
            for j in odd.any(1).nonzero().squeeze(1).tolist():  # what is not finite reaches the rows that see it
                o[see[:, j]] += torch.where(odd[j], v[j], 0)
            rows = slice(lo, lo + m), slice(h * grp, (h + 1) * grp)
            out[rows] = torch.where(some, o, 0)
            lse[rows] = torch.where(some, top + torch.log(over), -math.inf).squeeze(-1)
            # 32-bit scores move a weight by ds of itself; weights are rounded once to the cache's type
            ds = (dim + 4) * U32 * abs(scale) * (x.abs() @ k.abs().T).masked_fill(~at, 0).amax(-1, keepdim=True)
            steps = (see.sum(-1)[:, None, None] + 64) * U32
            mass = p @ v0.abs() / over
            small = flushed * torch.finfo(dtype).tiny * h16 * 2 * (at.double() @ v0.abs()) / over
            tol[rows] = h16 * o.abs() + 1.01 * (h16 + 2 * ds + steps) * mass + small
            lse_tol[rows] = torch.where(some, 2 * ds + steps + 2 * U32 * lse[rows].abs()[..., None], 0).squeeze(-1)
    return out, tol, lse, lse_tol
