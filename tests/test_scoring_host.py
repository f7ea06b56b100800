"""The operators between logits and ids, on the CPU: the library refuses bad
arguments before it touches a GPU, and so does the Python binding."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import byte_level_bpe_amd as B  # noqa: E402
from byte_level_bpe_amd import scoring  # noqa: E402

X = 1 << 20  # an aligned address that nothing reads
NAN, INF = float("nan"), float("inf")
MATRIX = [dict(dtype=3), dict(dtype=-1), dict(x=None), dict(x=X + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(n=1 << 31),
          dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(scale=1e-31), dict(scale=1e31)]
WRITTEN = [dict(dx=None), dict(dx=X + 1), dict(dstride=99), dict(dstride=0)]


def scores_call(**kw):
    a = dict(dtype=0, x=X, stride=100, n=3, vocab=100, ids=X, k=5, scale=1.0, lp=X, entropy=X, lse=X, ranks=X, top=X, top_lp=X, stats=X, ws=X, ws_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return scoring._lib().bbpe_token_logprobs(*a.values())


@pytest.mark.parametrize("bad", MATRIX + [dict(ids=None), dict(lp=None), dict(entropy=None), dict(lse=None), dict(ranks=None), dict(stats=None),
                                          dict(top=None), dict(top_lp=None), dict(k=257, vocab=1000), dict(k=101), dict(ids=X + 2),
                                          dict(stats=X + 4), dict(top=X + 1), dict(lse=X + 2)])
def test_scores_refuse(bad):
    assert scores_call(**bad) == B.E_INVALID_ARG


def test_scores_workspace():
    n = C.c_uint64()
    size, big = scoring._lib().bbpe_token_logprobs_workspace_bytes, dict(n=3, vocab=100000, stride=100000)
    assert size(0, 3, 100, 5, C.byref(n)) == 0 and n.value == 0 and size(0, 1 << 20, 100000, 5, C.byref(n)) == 0 and n.value == 0
    assert size(0, 3, 100000, 5, C.byref(n)) == 0 and n.value > 0
    assert scores_call(**big, ws=None) == B.E_WORKSPACE
    assert scores_call(**big, ws_bytes=n.value - 1) == B.E_WORKSPACE
    assert scores_call(**big, ws=X + 8) == B.E_WORKSPACE
    for bad in ((3, 3, 100, 5), (0, 1 << 31, 100, 5), (0, 3, 0, 0), (0, 3, 100, 101), (0, 3, 1000, 257)):
        assert size(*bad, C.byref(n)) == B.E_INVALID_ARG
    assert size(0, 3, 100, 5, None) == B.E_INVALID_ARG


def scores_back_call(**kw):
    a = dict(dtype=0, x=X, stride=100, n=3, vocab=100, ids=X, k=5, scale=1.0, entropy=X, top=X, stats=X, g=X, gh=X, gl=X, gt=X, dx=X, dstride=100,
             stream=None)
    a.update(kw)
    return scoring._lib().bbpe_token_logprobs_backward(*a.values())


@pytest.mark.parametrize("bad", MATRIX + WRITTEN + [dict(ids=None), dict(entropy=None), dict(stats=None), dict(top=None), dict(k=257, vocab=1000),
                                                    dict(gh=X + 1), dict(stats=X + 4)])
def test_scores_backward_refuses(bad):
    assert scores_back_call(**bad) == B.E_INVALID_ARG


def distill_call(**kw):
    a = dict(dtype=0, x=X, stride=100, n=3, vocab=100, ids=X, lp=X, k=5, tail=0, scale=1.0, loss=X, lse=X, stats=X, w=X, dx=X, dstride=100,
             ws=X, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return scoring._lib().bbpe_distill_loss(*a.values())


@pytest.mark.parametrize("bad", MATRIX + WRITTEN + [dict(ids=None), dict(lp=None), dict(k=0), dict(k=257, vocab=1000), dict(k=101), dict(k=100, tail=1),
                                                    dict(tail=2), dict(tail=-1), dict(loss=None), dict(lse=None), dict(stats=None), dict(w=None),
                                                    dict(stats=X + 8), dict(w=X + 2), dict(ids=X + 2)])
def test_distill_refuses(bad):
    assert distill_call(**bad) == B.E_INVALID_ARG


def test_distill_workspace():
    n = C.c_uint64()
    size, big = scoring._lib().bbpe_distill_loss_workspace_bytes, dict(n=3, vocab=100000, stride=100000, dstride=100000)
    assert size(0, 3, 100, C.byref(n)) == 0 and n.value == 0 and size(0, 1 << 20, 100000, C.byref(n)) == 0 and n.value == 0
    assert size(0, 3, 100000, C.byref(n)) == 0 and n.value > 0
    assert distill_call(**big, ws=None) == B.E_WORKSPACE
    assert distill_call(**big, ws_bytes=n.value - 1) == B.E_WORKSPACE
    assert distill_call(**big, ws=X + 8) == B.E_WORKSPACE
    for bad in ((3, 3, 100), (0, 1 << 31, 100), (0, 3, 0)):
        assert size(*bad, C.byref(n)) == B.E_INVALID_ARG
    assert size(0, 3, 100, None) == B.E_INVALID_ARG


def distill_back_call(**kw):
    a = dict(dtype=0, x=X, stride=100, n=3, vocab=100, ids=X, lp=X, k=5, tail=0, scale=1.0, stats=X, g=X, dx=X, dstride=100, stream=None)
    a.update(kw)
    return scoring._lib().bbpe_distill_loss_backward(*a.values())


@pytest.mark.parametrize("bad", MATRIX + WRITTEN + [dict(ids=None), dict(lp=None), dict(k=0), dict(k=100, tail=1), dict(stats=None), dict(g=None)])
def test_distill_backward_refuses(bad):
    assert distill_back_call(**bad) == B.E_INVALID_ARG


@pytest.mark.parametrize("call", [scores_back_call, distill_call, distill_back_call])
@pytest.mark.parametrize("across", [dict(dx=X + 2), dict(dx=X - 198), dict(dx=X + 200), dict(dstride=200), dict(stride=0), dict(dstride=-100),
                                    dict(stride=150, dstride=150, dx=X + 198), dict(stride=150, dstride=150, dx=X + 102), dict(stride=-100, dx=X),
                                    dict(n=1, stride=7, dstride=7, dx=X + 14), dict(stride=1 << 62, dx=X + 2)])
def test_gradients_across_the_logits_are_refused(call, across):
    assert call(**across) == B.E_INVALID_ARG


def test_no_rows_are_nothing_to_do():
    assert scores_call(n=0, x=None, ids=None) == 0 and scores_back_call(n=0, x=None, dx=None) == 0
    assert distill_call(n=0, x=None) == 0 and distill_back_call(n=0, x=None, dx=None) == 0


def refuses(call, says):
    with pytest.raises(B.BBPEError) as e:
        call()
    assert e.value.status == B.E_INVALID_ARG and says in str(e.value), str(e.value)


def test_python_refuses():
    """Host tensors, and what is wrong whatever the device."""
    x, ids = torch.zeros(3, 10), torch.zeros(3, dtype=torch.int32)
    top, lp, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.ones(3)
    scored = B.TokenLogprobs(w, w, w, ids, top, lp, torch.zeros(3, 2))
    found = B.DistillLoss(w, w, torch.zeros(3, 4))
    refuses(lambda: B.token_logprobs(x, ids), "tensors on a GPU")
    refuses(lambda: B.token_logprobs_backward(x, ids, scored, w), "tensors on a GPU")
    refuses(lambda: B.distill_loss(x, top, lp), "tensors on a GPU")
    refuses(lambda: B.distill_loss_backward(w, x, top, lp, found), "tensors on a GPU")
    for kw in (dict(weights=w), dict(dlogits=x)):
        refuses(lambda: B.distill_loss(x, top, lp, **kw), "given together")


def test_lost_gradients_are_refused():
    """Forms without a gradient refuse inputs that require one, unless grad mode is off."""
    x, ids = torch.zeros(3, 10, requires_grad=True), torch.zeros(3, dtype=torch.int32)
    top, lp, w = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.ones(3)
    scored = B.TokenLogprobs(w, w, w, ids, top, lp, torch.zeros(3, 2))
    found = B.DistillLoss(w, w, torch.zeros(3, 4))
    calls = [lambda: B.token_logprobs(x, ids, out=scored), lambda: B.distill_loss(x, top, lp, out=found),
             lambda: B.distill_loss(x, top, lp, weights=w, dlogits=torch.zeros(3, 10)),
             lambda: B.distill_loss(x.detach(), top, lp.clone().requires_grad_()),
             lambda: B.distill_loss(x.detach(), top, lp, weights=w.clone().requires_grad_(), dlogits=torch.zeros(3, 10))]
    for call in calls:
        refuses(call, "no_grad")
        with torch.no_grad():
            refuses(call, "tensors on a GPU")
