"""Outputs that a caller gives to the operators on torch tensors, on the GPU: they count as written, so that a backward
pass that has saved one of them raises instead of reading what is there now."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def lists():
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(5, 300, generator=g, device="cuda")
    ids = torch.tensor([1, 2, 3, 4, 299], dtype=torch.int32, device="cuda")
    return x, ids, B.token_logprobs(x, ids, top_k=4), torch.rand(5, generator=g, device="cuda")


@pytest.mark.parametrize("way", ["plain", "stream"])
def test_logits_that_become_their_gradient(way):
    """Scores recorded on the logits, which the one-call form then overwrites in place."""
    say("overwritten logits", way)
    x, ids, s, w = lists()
    leaf = x.clone().requires_grad_()
    how = dict(stream=torch.cuda.Stream()) if way == "stream" else {}
    for overwrite in (lambda y: B.distill_loss(y, s.top_ids, s.top_logprobs, weights=w, dlogits=y, **how),
                      lambda y: B.distill_loss_backward(w, y, s.top_ids, s.top_logprobs, B.distill_loss(y, s.top_ids, s.top_logprobs), dlogits=y, **how),
                      lambda y: B.token_logprobs_backward(y, ids, B.token_logprobs(y, ids), w, dlogits=y, **how)):
        for recorded in (lambda y: B.token_logprobs(y, ids).logprobs, lambda y: B.distill_loss(y, s.top_ids, s.top_logprobs).loss, torch.sin):
            y = leaf * 1.5
            out = recorded(y)
            torch.cuda.synchronize()
            overwrite(y.detach())
            torch.cuda.synchronize()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                out.sum().backward()
    say("into a tensor of its own: nothing is lost")
    y = leaf * 1.5
    out, other = B.token_logprobs(y, ids).logprobs, torch.empty_like(x)
    B.distill_loss(y.detach(), s.top_ids, s.top_logprobs, weights=w, dlogits=other, **how)
    torch.cuda.synchronize()
    out.sum().backward()
    assert other._version == 1 and bool(leaf.grad.any())


def test_given_outputs():
    say("given outputs")
    x, ids, s, w = lists()
    B.token_logprobs(x, ids, top_k=4, out=s)
    assert all(t._version == 1 for t in s)
    found = B.distill_loss(x, s.top_ids, s.top_logprobs)
    B.distill_loss(x, s.top_ids, s.top_logprobs, out=found)
    assert all(t._version == 1 for t in found)
    with torch.inference_mode():
        quiet = torch.empty_like(x)
    B.distill_loss(x, s.top_ids, s.top_logprobs, weights=w, dlogits=quiet)  # (keeps no versions)
    B.distill_loss_backward(w, x, s.top_ids, s.top_logprobs, found, dlogits=quiet)
    assert bool(quiet.isfinite().all())


def test_norm_and_attention():
    say("norm and attention")
    q, k = torch.randn(4, 4, 64, device="cuda", dtype=torch.bfloat16), torch.randn(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    pos, freq = torch.arange(4, device="cuda", dtype=torch.int32), torch.rand(16, device="cuda")
    leaf = q.clone().requires_grad_()
    y = leaf * 1.5
    out = B.qk_norm_rope(y, k, None, None, pos, freq)[0]
    B.qk_norm_rope(y.detach(), k, None, None, pos, freq, q_out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    dq, dk, attended = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    B.qk_norm_rope_backward(q, k, q, k, None, None, pos, freq, dq=dq, dk=dk)
    pages = torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    B.tree_attention(q, B.PagedCache(pages, torch.zeros_like(pages)), torch.zeros(1, 1, device="cuda", dtype=torch.int32),
                     torch.tensor([0, 4], device="cuda"), torch.zeros(1, device="cuda", dtype=torch.int32), out=attended)
    assert dq._version == dk._version == attended._version == 1
