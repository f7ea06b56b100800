"""Arguments of the operators between logits and ids that are not tensors, on the GPU: the short way and the long one take
the same."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import byte_level_bpe_amd as B  # noqa: E402
from tests.test_gpu_serving import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("scale", [0.5, 2, np.float32(0.5), np.float64(0.25), torch.tensor(0.5)])
@pytest.mark.parametrize("tail", [True, 2, 1, np.True_, False, 0, None])
def test_scales_and_tails(scale, tail):
    """What Python takes for a number or as true, on the current stream and on one that is given."""
    say("arguments", repr(scale), repr(tail))
    x = torch.randn(3, 300, generator=torch.Generator().manual_seed(1)).cuda()
    ids, w = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), torch.ones(3, device="cuda")
    results = []
    for how in (dict(), dict(stream=torch.cuda.Stream())):
        torch.cuda.synchronize()
        s = B.token_logprobs(x, ids, top_k=np.int64(4), scale=scale, **how)
        d = B.token_logprobs_backward(x, ids, s, w, scale=scale, **how)
        torch.cuda.synchronize()
        a = s.top_ids, s.top_logprobs
        found = B.distill_loss(x, *a, tail=tail, scale=scale, **how)
        e = B.distill_loss_backward(w, x, *a, found, tail=tail, scale=scale, **how)
        torch.cuda.synchronize()
        results.append([*s, d, *found, e])
    want = B.token_logprobs(x, ids, top_k=4, scale=float(scale))
    loss = B.distill_loss(x, want.top_ids, want.top_logprobs, tail=bool(tail), scale=float(scale)).loss
    for got in results:
        assert torch.equal(got[0], want.logprobs) and torch.equal(got[8], loss)
        assert all(torch.equal(p, q) for p, q in zip(got, results[0]))
