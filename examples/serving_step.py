"""From text to attention on one GPU: requests are encoded, their tokens placed
in a paged cache, prefilled, and a tree of drafted tokens is verified on top of
each; then one training step through the norm and the rotation.

    python examples/serving_step.py

The model is one attention layer with random weights: what the example shows is
how the calls fit together, and what stays on the device between them (ids,
offsets, pages, slots, positions: nothing is read back but the two plans'
status).
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import byte_level_bpe_amd as B  # noqa: E402

HQ, HK, DIM, PAGE = 8, 2, 64, 16


class Layer:
    """Embedding, one projection to queries, keys and values, and their norms' weights."""

    def __init__(self, vocab, g):
        dev, t = "cuda", torch.bfloat16
        self.emb = torch.randn(vocab, 256, generator=g, device=dev).to(t)
        self.w = (torch.randn(256, (HQ + 2 * HK) * DIM, generator=g, device=dev) / 16).to(t)
        self.wq = (1 + 0.1 * torch.randn(DIM, generator=g, device=dev)).to(t)
        self.wk = (1 + 0.1 * torch.randn(DIM, generator=g, device=dev)).to(t)
        self.inv_freq = torch.tensor([10000.0 ** (-2 * j / DIM) for j in range(DIM // 2)], device=dev)

    def qkv(self, ids):
        x = (self.emb[ids.long()] @ self.w).view(-1, HQ + 2 * HK, DIM)
        return x[:, :HQ], x[:, HQ:HQ + HK], x[:, HQ + HK:]

    def attend(self, ids, off, ctx, plan, cache, table, tree=None):
        q, k, v = self.qkv(ids)
        q, _ = B.qk_norm_rope(q, k, self.wq, self.wk, plan.positions, self.inv_freq, v=v, cache=cache, slots=plan.slots)
        return B.tree_attention(q, cache, table, off, ctx, tree_mask=tree)


def offsets(counts):
    out = torch.zeros(len(counts) + 1, dtype=torch.int64)
    out[1:] = torch.tensor(counts).cumsum(0)
    return out.cuda()


def ancestors(parents):
    """Mask words and depths of one tree: parents[i] < i, -1 for a root."""
    words, depth = [], []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return words, depth


def main():
    from synth import configs
    w = configs.tiny()
    tok = B.load_ranks(w.tokens, w.specials, w.grammar)
    text = w.segments[0][0]
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = Layer(tok.info()["max_id"] + 1, g)
    cache = B.PagedCache(*(torch.zeros(256, HK, PAGE, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    free = torch.randperm(256, generator=g, device="cuda").to(torch.int32)

    # prompts: encode, place, prefill
    prompts = [text[:400], text[400:430], text[430:1500]]
    data, seg_off, allow, total = B.to_device_segments([(p, False) for p in prompts])
    ids, off, n = tok.encode_device(data, seg_off, allow, total)
    ctx = torch.zeros(len(prompts), dtype=torch.int32, device="cuda")
    table = torch.full((len(prompts), 64), -1, dtype=torch.int32, device="cuda")
    plan = B.block_tables(off, ctx, free, table, PAGE, n)
    layer.attend(ids, off, ctx, plan, cache, table)
    taken, _ = plan.wait()
    print("prompts: %d tokens in %d pages" % (n, taken))

    # a tree of drafts for each: two continuations of the first draft, one of which goes on
    parents = [-1, 0, 0, 1, 3]
    words, depth = ancestors(parents)
    ctx, m = plan.seq_len.clone(), len(parents)
    drafts = torch.randint(0, 256, (len(prompts) * m,), generator=g, device="cuda", dtype=torch.int32)
    off = offsets([m] * len(prompts))
    mask = torch.tensor(words * len(prompts), dtype=torch.int64, device="cuda")[:, None]
    plan = B.block_tables(off, ctx, free[taken:].contiguous(), table, PAGE, len(drafts),
                          depth=torch.tensor(depth * len(prompts), dtype=torch.int32, device="cuda"))
    tree = layer.attend(drafts, off, ctx, plan, cache, table, mask)
    more, _ = plan.wait()
    print("drafts: %d nodes on contexts of %s tokens, %d more pages" % (len(drafts), ctx.tolist(), more))

    # the path 0, 1, 3, 4 again as a chain, as if it had been accepted: the same rows
    path = [0, 1, 3, 4]
    chain_ids = drafts.view(-1, m)[:, path].reshape(-1).contiguous()
    chain_off = offsets([len(path)] * len(prompts))
    plan = B.block_tables(chain_off, ctx, free[taken:].contiguous(), table, PAGE, len(chain_ids))
    chain = layer.attend(chain_ids, chain_off, ctx, plan, cache, table)
    plan.wait()
    off_by = (tree.view(-1, m, HQ, DIM)[:, path].reshape(chain.shape).float() - chain.float()).abs().max().item()
    print("the accepted path as a chain differs by at most %.2g" % off_by)

    # training: gradients through the norm and the rotation
    q, k, _ = layer.qkv(chain_ids)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, layer.wq, layer.wk)]
    out = B.qk_norm_rope(*leaves, plan.positions, layer.inv_freq)
    loss = sum((o.float() * torch.randn(o.shape, generator=g, device="cuda")).sum() for o in out)
    loss.backward()
    print("gradient norms: " + ", ".join("%.3g" % t.grad.float().norm().item() for t in leaves))
    return off_by, tree, leaves


if __name__ == "__main__":
    main()
