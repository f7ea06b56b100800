"""What the outputs of the operators between logits and ids keep in memory, on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402

BLOCK = 512  # the allocator's smallest: a tensor by itself takes as much


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("way", ["plain", "stream", "recorded"])
@pytest.mark.parametrize("n,k", [(0, 0), (1, 0), (1, 20), (8, 5), (8, 6), (9, 5), (21, 0), (22, 0), (700, 0), (700, 20)])
def test_outputs_keep_no_others(n, k, way):
    """One that is kept when the others are dropped holds on to its own bytes, or to a block of the allocator's."""
    say("storage", n, k, way)
    x = torch.randn(n, 300, device="cuda", requires_grad=way == "recorded")
    ids = torch.arange(n, dtype=torch.int32) % 300
    how = dict(stream=torch.cuda.Stream()) if way == "stream" else {}
    ids_there = ids.cuda()
    torch.cuda.synchronize()
    got = B.token_logprobs(x, ids_there, top_k=k, **how)
    outs = list(got)
    if k:
        outs += list(B.distill_loss(x, got.top_ids, got.top_logprobs.detach(), **how))
    torch.cuda.synchronize()
    for t in outs:
        size = t.numel() * t.element_size()
        assert t.untyped_storage().nbytes() <= max(BLOCK, size + 15), (t.shape, t.untyped_storage().nbytes())
        assert t.is_contiguous() and t.device == x.device and (not t.numel() or t.data_ptr() % 16 == 0)
    want = torch.log_softmax(x.detach().cpu().double(), 1).gather(1, ids.long()[:, None])[:, 0]
    assert bool(((got.logprobs.detach().cpu() - want).abs() < 1e-5).all()) and got.top_ids.shape == (n, k)


def test_collected_scores():
    """Four bytes a token of a long run, and no more: 64 steps of 4,096 rows."""
    say("collected")
    x, ids = torch.randn(4096, 40, device="cuda"), torch.zeros(4096, device="cuda", dtype=torch.int32)
    B.token_logprobs(x, ids, top_k=4)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [B.token_logprobs(x, ids, top_k=4).logprobs for _ in range(64)]
    assert torch.cuda.memory_allocated() - before == 64 * 4096 * 4
    lists = [B.token_logprobs(x, ids, top_k=4).top_ids for _ in range(64)]
    assert torch.cuda.memory_allocated() - before == 64 * 4096 * 4 * 5
    losses = [B.distill_loss(x, t, torch.zeros(4096, 4, device="cuda")).loss for t in lists]
    assert torch.cuda.memory_allocated() - before == 64 * 4096 * 4 * 6
    del kept, lists, losses
    assert torch.cuda.memory_allocated() == before


def test_outputs_by_themselves():
    """Each can be written, resized by a copy and freed without the others: versions, streams and allocator know it."""
    say("by themselves")
    x, ids = torch.randn(600, 50, device="cuda"), torch.zeros(600, device="cuda", dtype=torch.int32)
    for n in (3, 600):
        got = B.token_logprobs(x[:n], ids[:n], top_k=3)
        want = [t.clone() for t in got]
        got.logprobs.fill_(7.0)
        got.stats.record_stream(torch.cuda.Stream())
        assert got.logprobs._version == 1 and got.entropy._version == 0
        assert all(torch.equal(a, b) for a, b in zip(list(got)[1:], want[1:])) and bool((got.logprobs == 7).all())
        with torch.inference_mode():
            quiet = B.token_logprobs(x[:n], ids[:n], top_k=3)
            assert all(t.is_inference() for t in quiet) and all(torch.equal(a, b) for a, b in zip(quiet, want))
