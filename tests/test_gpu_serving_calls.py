"""What calls of the operators between ids and attention keep, and refuse, on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tables_args(tokens, n=2, page=16):
    dev = "cuda"
    off = torch.tensor([0] + [tokens] * n, dtype=torch.int64, device=dev)
    width = -(-tokens // page) + 1
    return (off, torch.zeros(n, dtype=torch.int32, device=dev), torch.arange(width, dtype=torch.int32, device=dev),
            torch.zeros(n, width, dtype=torch.int32, device=dev), page)


@pytest.mark.parametrize("on_a_stream", [False, True])
def test_lengths_do_not_keep_the_tokens_outputs(on_a_stream):
    """seq_len is the next step's ctx_len: what it holds on to is a request's size, not a token's."""
    say("storage", on_a_stream)
    args = tables_args(5000)
    torch.cuda.synchronize()
    plan = B.block_tables(*args, 5000, **(dict(stream=torch.cuda.Stream()) if on_a_stream else {}))
    torch.cuda.synchronize()
    assert plan.seq_len.tolist() == [5000, 0] and plan.wait() == (313, 5000)
    assert max(t.untyped_storage().nbytes() for t in (plan.seq_len, plan.status)) < 1000
    assert all(t.data_ptr() % 16 == 0 for t in plan)


@pytest.mark.parametrize("tokens,page", [(1 << 31, 16), (1 << 40, 16), (1 << 62, 16), (-1, 16), (5, 0), (5, -16), (5, (1 << 30) + 1), (5, 1 << 32)])
def test_sizes_are_refused_before_memory_is_taken(tokens, page):
    say("sizes", tokens, page)
    args = tables_args(5)[:4]
    for kw in ({}, dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(B.BBPEError) as e:
            B.block_tables(*args, page, tokens, **kw)
        assert e.value.status == B.E_INVALID_ARG
