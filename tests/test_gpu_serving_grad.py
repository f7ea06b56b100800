"""Gradients through qk_norm_rope, as training code meets them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests import serving_reference as ref  # noqa: E402
from tests.test_gpu_serving import near, norm_inputs, say  # noqa: E402

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("n,hq,hk,dim,rot,dtype,inter", [(7, 4, 2, 64, 64, BF, False), (5, 3, 1, 128, 64, HF, True), (9, 2, 2, 80, 32, F, False),
                                                         (1, 1, 1, 16, 16, BF, True)])
@pytest.mark.parametrize("weights", [True, False])
def test_gradients(n, hq, hk, dim, rot, dtype, inter, weights):
    """Against the gradient's formula in 64 bits; the weights' once more rounded, to their type."""
    say("grad", n, hq, hk, dim, rot, dtype, inter, weights)
    wide, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, rot, dtype, 17)
    x = dev.clone().requires_grad_()
    ws = [t.cuda().requires_grad_() for t in w] if weights else [None, None]
    q, k = B.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], *ws, pos.cuda(), freq.cuda(), eps=1e-5, interleaved=inter)
    near(q.detach(), *ref.norm_rope(wide[:, :hq], w[0] if weights else None, pos, freq, 1e-5, inter), "q")
    gq, gk = torch.randn(n, hq, dim, generator=g).to(dtype), torch.randn(n, hk, dim, generator=g).to(dtype)
    torch.autograd.backward([q, k], [gq.cuda(), gk.cuda()])
    for lo, hi, up, ww, leaf in ((0, hq, gq, w[0], ws[0]), (hq, hq + hk, gk, w[1], ws[1])):
        (dx, tol), (dw, wtol) = ref.norm_rope_grad(up, wide[:, lo:hi], ww if weights else None, pos, freq, 1e-5, inter)
        near(x.grad[:, lo:hi], dx, tol, "dx")
        if weights:
            assert leaf.grad.dtype is dtype
            tiny = torch.finfo(dtype).tiny * ref.half_step(dtype) * 2
            near(leaf.grad, dw, (1 + ref.half_step(dtype)) * wtol + ref.half_step(dtype) * dw.abs() + tiny, "dw")
    assert not x.grad[:, hq + hk:].any()


def test_gradients_of_a_sum_of_one_output_and_on_a_stream():
    """A gradient broadcast over every dimension, an output that is not used, one weight that is not trained; and on
    another stream the same bits."""
    say("sum")
    n, hq, hk, dim = 6, 4, 2, 64
    wide, dev, w, pos, freq, _ = norm_inputs(n, hq, hk, dim, dim, F, 19)
    got = []
    for stream in (None, torch.cuda.Stream()):
        x, wq, wk = dev.clone().requires_grad_(), w[0].cuda().requires_grad_(), w[1].cuda()
        torch.cuda.synchronize()
        q, k = B.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], wq, wk, pos.cuda(), freq.cuda(), stream=stream)
        torch.cuda.synchronize()
        q.sum().backward()
        torch.cuda.synchronize()
        assert wk.grad is None and not x.grad[:, hq:].any()
        got.append((x.grad, wq.grad))
    (dx, tol), (dw, wtol) = ref.norm_rope_grad(torch.ones(n, hq, dim), wide[:, :hq], w[0], pos, freq, 1e-6, False)
    near(got[0][0][:, :hq], dx, tol, "dx")
    near(got[0][1], dw, wtol, "dw")
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_gradients_only_where_wanted():
    say("no grad")
    n, hq, hk, dim = 3, 2, 1, 32
    _, dev, w, pos, freq, _ = norm_inputs(n, hq, hk, dim, dim, BF, 23)
    a = [dev[:, :hq], dev[:, hq:hq + hk], w[0].cuda().requires_grad_(), w[1].cuda(), pos.cuda(), freq.cuda()]
    with torch.no_grad():
        assert not any(t.requires_grad for t in B.qk_norm_rope(*a))
    assert all(t.requires_grad for t in B.qk_norm_rope(*a))
    plain = [t.detach() for t in a]
    assert not any(t.requires_grad for t in B.qk_norm_rope(*plain))
    assert all(torch.equal(x, y) for x, y in zip(B.qk_norm_rope(*a), B.qk_norm_rope(*plain)))
    say("inputs changed between the passes, and a second derivative, are refused")
    q, _ = B.qk_norm_rope(*a)
    with torch.no_grad():
        a[2].mul_(2)
    with pytest.raises(RuntimeError):
        q.sum().backward()
    (dw,) = torch.autograd.grad(B.qk_norm_rope(*a)[0].float().square().sum(), a[2], create_graph=True)
    with pytest.raises(RuntimeError):
        dw.sum().backward()
    say("the backward kernel by itself takes inputs that require grad")
    assert len(B.qk_norm_rope_backward(torch.ones(n, hq, dim, dtype=BF, device="cuda"), torch.ones(n, hk, dim, dtype=BF, device="cuda"), *a)) == 4


def test_gradients_in_a_graph():
    """Forward and backward captured together and replayed, with other inputs and eager passes between."""
    say("graph")
    n, hq, hk, dim = 700, 4, 2, 64
    _, dev, w, pos, freq, g = norm_inputs(n, hq, hk, dim, dim, BF, 37)
    x, ws = dev.clone().requires_grad_(), [t.cuda().requires_grad_() for t in w]
    up = [torch.randn(n, h, dim, generator=g).to(BF).cuda() for h in (hq, hk)]
    pos, freq = pos.cuda(), freq.cuda()

    def step():
        out = B.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], *ws, pos, freq)
        grads = torch.autograd.grad(out, (x, *ws), up)
        return [t.detach() for t in out] + list(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        with torch.no_grad():
            x.mul_(1.25)
            up[0].add_(0.5)
            ws[1].neg_()
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
