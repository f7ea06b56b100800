"""Calls of the operators between ids and attention that the Python binding has
to refuse before it looks at a device: on the CPU, told apart by what they say."""
import pytest

torch = pytest.importorskip("torch")

import byte_level_bpe_amd as B  # noqa: E402

BF = torch.bfloat16


def refuses(call, says):
    with pytest.raises(B.BBPEError) as e:
        call()
    assert e.value.status == B.E_INVALID_ARG and says in str(e.value), str(e.value)


def norm_args(grad=()):
    q, k, wq, wk = (torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 2, 64, dtype=BF), torch.ones(64, dtype=BF), torch.ones(64, dtype=BF))
    for t in (t for name, t in zip(("q", "k", "wq", "wk"), (q, k, wq, wk)) if name in grad):
        t.requires_grad_()
    return q, k, wq, wk, torch.zeros(3, dtype=torch.int32), torch.zeros(32)


def cache():
    return B.PagedCache(torch.zeros(4, 2, 16, 64, dtype=BF), torch.zeros(4, 2, 16, 64, dtype=BF))


def test_norm_into_a_cache_wants_all_of_it():
    """Without a cache, values and slots would be dropped and nothing stored."""
    v, slots, c = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, dtype=torch.int64), cache()
    for kw in (dict(slots=slots), dict(v=v), dict(v=v, slots=slots), dict(cache=c), dict(cache=c, v=v), dict(cache=c, slots=slots)):
        refuses(lambda: B.qk_norm_rope(*norm_args(), **kw), "given together")
    refuses(lambda: B.qk_norm_rope(*norm_args(), cache=c, v=v, slots=slots), "tensors on a GPU")
    refuses(lambda: B.qk_norm_rope(*norm_args()), "tensors on a GPU")


@pytest.mark.parametrize("grad", ["q", "k", "wq", "wk"])
def test_lost_gradients_are_refused(grad):
    """Forms without a gradient refuse inputs that require one, unless grad mode is off."""
    v, slots, c = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(3, dtype=torch.int64), cache()
    a = norm_args((grad,))
    refuses(lambda: B.qk_norm_rope(*a, cache=c, v=v, slots=slots), "no_grad")
    refuses(lambda: B.qk_norm_rope(*a, q_out=torch.zeros(3, 4, 64, dtype=BF)), "no_grad")
    refuses(lambda: B.qk_norm_rope(*a, k_out=torch.zeros(3, 2, 64, dtype=BF)), "no_grad")
    refuses(lambda: B.qk_norm_rope(*a[:5], a[5].clone().requires_grad_()), "no_grad")
    table, off, ctx = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    attend = lambda: B.tree_attention(a[0], c, table, off, ctx)  # noqa: E731
    refuses(attend, "no_grad" if grad == "q" else "tensors on a GPU")
    with torch.no_grad():
        refuses(lambda: B.qk_norm_rope(*a, cache=c, v=v, slots=slots), "tensors on a GPU")
        refuses(attend, "tensors on a GPU")


def test_a_paged_cache_is_fixed():
    """Its description for the kernels is made once: another tensor in its place would leave them at the old memory."""
    c = cache()
    p, k = c._p, c.k
    for name in ("k", "v", "page_size", "n_pages", "dtype", "_s", "_p"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    assert c._p == p and c.k is k
    c.layer = 3  # a program's own
    assert c.layer == 3
