"""The operators between ids and attention, on the CPU: the library refuses bad
arguments before it touches a GPU, and so does the Python binding."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import byte_level_bpe_amd as B  # noqa: E402
from byte_level_bpe_amd import serving  # noqa: E402

X = 1 << 20  # an aligned address that nothing reads


def cache(**kw):
    c = dict(k=X, v=X, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, dtype=0, page_stride=2048, head_stride=1024,
             token_stride=64)
    c.update(kw)
    return serving._CacheStruct(*(c[n] for n, _ in serving._CacheStruct._fields_))


def tables_call(**kw):
    a = dict(q_off=X, ctx=X, n=2, free=X, n_free=4, table=X, stride=8, width=8, page=16, tokens=0, depth=None, slots=X, pos=X,
             req=X, seq=X, status=X, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return serving._lib().bbpe_block_tables(*a.values())


@pytest.mark.parametrize("bad", [dict(q_off=None), dict(ctx=None), dict(free=None), dict(table=None), dict(status=None),
                                 dict(seq=None), dict(tokens=5, slots=None), dict(tokens=5, pos=None), dict(page=0),
                                 dict(stride=7), dict(n_free=1 << 31), dict(tokens=1 << 31), dict(n=(1 << 24) + 1),
                                 dict(width=1 << 31), dict(q_off=X + 4), dict(ctx=X + 2), dict(slots=X + 4, tokens=1),
                                 dict(page=(1 << 30) + 1)])
def test_block_tables_refuses(bad):
    assert tables_call(**bad) == B.E_INVALID_ARG


def test_block_tables_workspace():
    n = C.c_uint64()
    lib = serving._lib()
    assert lib.bbpe_block_tables_workspace_bytes(4096, C.byref(n)) == 0 and n.value == 0
    assert lib.bbpe_block_tables_workspace_bytes(4097, C.byref(n)) == 0 and n.value >= 4 * 4097
    assert lib.bbpe_block_tables_workspace_bytes(1, None) == B.E_INVALID_ARG
    assert tables_call(n=4097) == B.E_WORKSPACE
    assert tables_call(n=4097, ws=X, ws_bytes=n.value - 1) == B.E_WORKSPACE
    assert tables_call(n=4097, ws=X + 8, ws_bytes=n.value) == B.E_WORKSPACE


def norm_call(**kw):
    a = dict(dtype=0, n=3, hq=4, hk=2, dim=64, rot=64, inter=0, eps=1e-6, q=X, qt=256, qh=64, k=X, kt=128, kh=64, v=None, vt=0,
             vh=0, wq=X, wk=X, pos=X, freq=X, qo=X, qot=256, qoh=64, ko=X, kot=128, koh=64, cache=None, slots=None, stream=None)
    a.update(kw)
    return serving._lib().bbpe_qk_norm_rope(*a.values())


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(dim=0), dict(dim=72), dict(dim=272), dict(rot=80), dict(rot=24),
                                 dict(inter=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None), dict(k=None), dict(qo=None),
                                 dict(ko=None), dict(pos=None), dict(freq=None), dict(wq=X + 2), dict(q=X + 1), dict(hq=0, hk=0),
                                 dict(hq=5000), dict(slots=X), dict(n=1 << 31), dict(pos=X + 2)])
def test_norm_refuses(bad):
    assert norm_call(**bad) == B.E_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(page_size=0), dict(head_dim=128), dict(n_kv_heads=3), dict(dtype=1), dict(k=None), dict(v=X + 8),
                                 dict(token_stride=60), dict(page_stride=2049), dict(n_pages=1 << 31)])
def test_norm_refuses_caches(bad):
    ok = cache()
    assert norm_call(cache=C.addressof(ok)) == B.E_INVALID_ARG  # no slots
    assert norm_call(cache=C.addressof(ok), slots=X) == B.E_INVALID_ARG  # no v
    c = cache(**bad)
    assert norm_call(cache=C.addressof(c), slots=X, v=X, vt=128, vh=64) == B.E_INVALID_ARG


def back_call(**kw):
    a = dict(dtype=0, n=3, hq=4, hk=2, dim=64, rot=64, inter=0, eps=1e-6, gq=X, gqt=256, gqh=64, gk=X, gkt=128, gkh=64, q=X, qt=256,
             qh=64, k=X, kt=128, kh=64, wq=X, wk=X, pos=X, freq=X, dq=X, dqt=256, dqh=64, dk=X, dkt=128, dkh=64, dwq=X, dwk=X, ws=X,
             ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return serving._lib().bbpe_qk_norm_rope_backward(*a.values())


def test_norm_backward_refuses():
    for bad in (dict(gq=None), dict(gk=None), dict(dq=None), dict(dk=None), dict(dim=40), dict(dwq=X + 1), dict(q=None)):
        assert back_call(**bad) == B.E_INVALID_ARG, bad
    n = C.c_uint64()
    assert serving._lib().bbpe_qk_norm_rope_backward_workspace_bytes(3, 64, C.byref(n)) == 0
    assert back_call(ws=None) == B.E_WORKSPACE
    assert back_call(ws_bytes=n.value - 1) == B.E_WORKSPACE
    assert back_call(ws=X + 16) == B.E_WORKSPACE


def attn_call(c=None, **kw):
    c = cache() if c is None else c
    a = dict(q=X, qt=256, qh=64, n=3, hq=4, cache=C.addressof(c), table=X, stride=8, width=8, q_off=X, ctx=X, n_req=2, mask=None,
             words=0, scale=0.125, out=X, ot=256, oh=64, lse=X, ws=X, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return serving._lib().bbpe_tree_attention(*a.values())


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(table=None), dict(q_off=None), dict(ctx=None), dict(width=0),
                                 dict(hq=3), dict(hq=0), dict(hq=258), dict(mask=X), dict(scale=float("inf")),
                                 dict(scale=float("nan")), dict(stride=7), dict(width=1 << 27, stride=1 << 27), dict(q=X + 1),
                                 dict(lse=X + 2), dict(mask=X + 4, words=1), dict(cache=None), dict(n=1 << 31)])
def test_attention_refuses(bad):
    assert attn_call(**bad) == B.E_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(head_dim=96), dict(page_size=4), dict(page_size=24), dict(page_size=1 << 17),
                                 dict(n_kv_heads=0), dict(n_pages=0), dict(k=None), dict(k=X + 2), dict(head_stride=1023)])
def test_attention_refuses_caches(bad):
    assert attn_call(cache(**bad)) == B.E_INVALID_ARG
    n = C.c_uint64()
    c = cache(**bad)
    assert serving._lib().bbpe_tree_attention_workspace_bytes(3, 2, 4, C.addressof(c), C.byref(n)) == B.E_INVALID_ARG


def test_attention_workspace():
    n, c = C.c_uint64(), cache()
    assert serving._lib().bbpe_tree_attention_workspace_bytes(3, 2, 4, C.addressof(c), C.byref(n)) == 0
    assert attn_call(ws=None) == B.E_WORKSPACE
    assert attn_call(ws_bytes=n.value - 1) == B.E_WORKSPACE
    assert attn_call(ws=X + 8) == B.E_WORKSPACE
    assert attn_call(n=0) == 0 and attn_call(n_req=0) == 0  # nothing to do


def test_python_refuses_host_tensors_and_shapes():
    i32, i64 = torch.int32, torch.int64
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, freq = torch.zeros(3, dtype=i32), torch.zeros(32)
    table, off, ctx = torch.zeros(2, 4, dtype=i32), torch.zeros(3, dtype=i64), torch.zeros(2, dtype=i32)
    c = B.PagedCache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    for call in (lambda: B.qk_norm_rope(q, k, None, None, pos, freq),
                 lambda: B.qk_norm_rope_backward(q, k, q, k, None, None, pos, freq),
                 lambda: B.block_tables(off, ctx, torch.zeros(4, dtype=i32), table, 16, 3),
                 lambda: B.tree_attention(q, c, table, off, ctx)):
        with pytest.raises(B.BBPEError) as e:
            call()
        assert e.value.status == B.E_INVALID_ARG
    for kv in ((torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64)),
               (torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)),
               (torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 8, 64, dtype=torch.float16)),
               (torch.zeros(4, 2, 16, 65, dtype=torch.float16)[..., :64], torch.zeros(4, 2, 16, 65, dtype=torch.float16)[..., :64]),
               (torch.zeros(4, 2, 64, dtype=torch.float16), torch.zeros(4, 2, 64, dtype=torch.float16))):
        with pytest.raises(B.BBPEError) as e:
            B.PagedCache(*kv)
        assert e.value.status == B.E_INVALID_ARG
