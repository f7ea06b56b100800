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
