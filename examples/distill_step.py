"""From text to a distillation step on one GPU: requests are encoded, their tokens
scored by a teacher (log probabilities, entropies and the most likely
alternatives of every next token), and a smaller student is trained one step on
the alternatives.

    python examples/distill_step.py

Teacher and student are a table of embeddings and one matrix each, with random
weights: what the example shows is how the calls fit together, and that
everything between text and gradients stays on the device.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import byte_level_bpe_amd as B  # noqa: E402

TOP, SCALE = 32, 1 / 1.5  # alternatives a token, 1 / temperature


def model(vocab, width, g):
    """Embeddings and the matrix to logits."""
    emb = torch.randn(vocab, width, generator=g, device="cuda")
    head = torch.randn(width, vocab, generator=g, device="cuda") * 3 / width ** 0.5
    return emb.to(torch.bfloat16), head.to(torch.bfloat16)


def main():
    from synth import configs
    w = configs.tiny()
    tok = B.load_ranks(w.tokens, w.specials, w.grammar)
    text = w.segments[0][0]
    vocab = tok.info()["max_id"] + 1
    g = torch.Generator(device="cuda").manual_seed(0)
    requests = [text[:400], text[400:430], text[430:1500]]
    data, seg_off, allow, total = B.to_device_segments([(r, False) for r in requests])
    ids, off, n = tok.encode_device(data, seg_off, allow, total)

    # the token after each; the last of a request has none
    after = torch.cat([ids[1:n], ids.new_full((1,), -1)])
    after[off[1:] - 1] = -1

    # the teacher's side: scores of the text, and what it would have said instead
    emb, head = model(vocab, 256, g)
    scored = B.token_logprobs(emb[ids[:n].long()] @ head, after, top_k=TOP, scale=SCALE)
    print("%d tokens: mean log probability %.3f, mean entropy %.3f, mean rank %.0f" %
          (n, scored.logprobs.mean().item(), scored.entropy.mean().item(), scored.ranks.float().mean().item()))
    # tokens without a next one are left out: a list that ends at once
    lists = scored.top_ids.masked_fill((after < 0)[:, None], -1)

    # the student's: a step with gradients recorded
    leaves = [t.requires_grad_() for t in model(vocab, 64, g)]
    logits = leaves[0][ids[:n].long()] @ leaves[1]
    loss = B.distill_loss(logits, lists, scored.top_logprobs, tail=True, scale=SCALE).loss
    loss.sum().div(n).backward()

    # the same in one call, the gradient in place of the logits
    with torch.no_grad():
        again = leaves[0][ids[:n].long()] @ leaves[1]
        both = B.distill_loss(again, lists, scored.top_logprobs, tail=True, scale=SCALE,
                              weights=torch.full((n,), 1.0 / n, device="cuda"), dlogits=again)
    print("loss %.4f; gradient norms: %s; in one call: loss %.4f, gradient norm of the logits %.3g" % (
        loss.mean().item(), ", ".join("%.3g" % t.grad.float().norm().item() for t in leaves), both.loss.mean().item(),
        again.float().norm().item()))
    return scored, (loss.detach(), both.loss), leaves


if __name__ == "__main__":
    main()
