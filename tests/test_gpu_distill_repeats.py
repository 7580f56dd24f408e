"""The same inputs give the same bits, with lists that name tokens twice from entries that
different warps take."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from test_gpu_logits import _check_distill, _logits  # noqa: E402

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


# several CTAs a row, one of 256 threads, of 128, of 64
@pytest.mark.parametrize("N,V", [(9, 90001), (1500, 20000), (310, 5000), (2500, 2000)])
@pytest.mark.parametrize("K", [80, 300])
def test_doubly_listed_tokens_give_the_same_bits_every_time(N, V, K):
    rng = np.random.default_rng(K)
    z = _logits(rng, N, V, torch.float32).contiguous()
    idx = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    idx[:, 40:80] = idx[:, :40]        # entries of another warp
    idx[:, 33] = idx[:, 1]             # three times
    if K > 200:
        idx[:, 260:300] = idx[:, :40]  # entries of a thread's second turn
    lab = idx[:, 5].copy()
    idx, val = torch.from_numpy(idx).cuda(), torch.from_numpy(rng.normal(0, 1, (N, K)).astype(np.float32)).cuda()
    for k in (2, 3):                   # and masked
        z[torch.arange(0, N, 4, device="cuda"), idx[::4, k].long()] = -INF
    masked = torch.isinf(torch.gather(z, 1, idx.long()))
    val = torch.where(masked, -INF, val)  # so that the loss stays finite
    rest = torch.zeros(N, device="cuda")
    labels = torch.from_numpy(lab).cuda()
    op = tw.DistillLoss(N, V, K, dtype=torch.float32, temperature=1.5, kd_weight=0.5, ce_weight=0.5)
    loss, dz = (t.clone() for t in op.forward_backward(z, idx, val, rest=rest, labels=labels))
    few = torch.tensor([0, 1, 4, N - 1], device="cuda")
    _check_distill(loss[few], dz[few], z[few], idx[few], val[few], rest[few], labels[few], 1.5, 0.5, 0.5)
    for _ in range(60):
        l2, d2 = op.forward_backward(z, idx, val, rest=rest, labels=labels)
        assert torch.equal(l2, loss) and torch.equal(d2, dz)
