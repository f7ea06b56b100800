"""Inputs of forward-mode differentiation, on the GPU: the operators on torch tensors have no forward gradients and say
so, instead of returning outputs without their tangents."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from torch.autograd import forward_ad  # noqa: E402

import byte_level_bpe_amd as B  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def refuses(call):
    with pytest.raises(B.BBPEError) as e:
        call()
    assert e.value.status == B.E_INVALID_ARG and "tangent" in str(e.value)


def scoring():
    n, v, k = 3, 40, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    x, ids = torch.randn(n, v, generator=g, device="cuda"), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    s = B.token_logprobs(x, ids, top_k=k)
    return x, ids, s, torch.ones(n, device="cuda"), torch.ones(n, k, device="cuda")


def test_scores_and_distillation():
    say("scores and distillation")
    x, ids, s, w, wk = scoring()
    found = B.distill_loss(x, s.top_ids, s.top_logprobs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for kw in (dict(), dict(stream=side)):
            refuses(lambda: B.token_logprobs(dual(x), ids, **kw))
            refuses(lambda: B.token_logprobs_backward(x, ids, s, dual(w), **kw))
            refuses(lambda: B.token_logprobs_backward(dual(x), ids, s, w, **kw))
            refuses(lambda: B.token_logprobs_backward(x, ids, s, grad_top=dual(wk), **kw))
            refuses(lambda: B.distill_loss(dual(x), s.top_ids, s.top_logprobs, **kw))
            refuses(lambda: B.distill_loss(x, s.top_ids, dual(s.top_logprobs), **kw))
            refuses(lambda: B.distill_loss(x, s.top_ids, s.top_logprobs, weights=dual(w), dlogits=torch.empty_like(x), **kw))
            refuses(lambda: B.distill_loss_backward(dual(w), x, s.top_ids, s.top_logprobs, found, **kw))
        refuses(lambda: B.token_logprobs(dual(x), ids, out=s))
        with torch.no_grad():
            refuses(lambda: B.token_logprobs(dual(x), ids))
        leaf = x.clone().requires_grad_()
        refuses(lambda: B.token_logprobs(dual(leaf), ids))
        say("a tangent of the gradient that comes back")
        for out in (B.token_logprobs(leaf, ids).logprobs, B.distill_loss(leaf, s.top_ids, s.top_logprobs).loss):
            refuses(lambda: torch.autograd.grad(out, leaf, dual(w), retain_graph=True))
            assert torch.autograd.grad(out, leaf, w)[0].isfinite().all()
        say("what carries none is taken, and so is what has been unpacked")
        again = B.token_logprobs(forward_ad.unpack_dual(dual(x)).primal, ids, top_k=4)
        assert all(torch.equal(a, b) for a, b in zip(again, s))
        with torch.inference_mode():
            assert torch.equal(B.token_logprobs(x, ids).logprobs, s.logprobs)


def test_norm_and_attention():
    say("norm and attention")
    q, k = torch.randn(4, 4, 64, device="cuda", dtype=torch.bfloat16), torch.randn(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    pos, freq = torch.arange(4, device="cuda", dtype=torch.int32), torch.rand(16, device="cuda")
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    pages = torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    cache = B.PagedCache(pages, torch.zeros_like(pages))
    table = torch.zeros(1, 1, device="cuda", dtype=torch.int32)
    off, ctx = torch.tensor([0, 4], device="cuda"), torch.zeros(1, device="cuda", dtype=torch.int32)
    want = B.qk_norm_rope(q, k, w, w, pos, freq)
    torch.cuda.synchronize()
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        refuses(lambda: B.qk_norm_rope(dual(q), k, w, w, pos, freq))
        refuses(lambda: B.qk_norm_rope(q, k, w, dual(w), pos, freq))
        refuses(lambda: B.qk_norm_rope(q, k, w, w, pos, dual(freq)))
        refuses(lambda: B.qk_norm_rope_backward(dual(q), k, q, k, w, w, pos, freq))
        refuses(lambda: B.tree_attention(dual(q), cache, table, off, ctx))
        assert all(torch.equal(a, b) for a, b in zip(B.qk_norm_rope(q, k, w, w, pos, freq), want))
        assert B.tree_attention(q, cache, table, off, ctx).shape == q.shape
