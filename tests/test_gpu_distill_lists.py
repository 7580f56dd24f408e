"""Teacher lists that name a token many times: each entry is a term of the sum, whichever of
them meets the token's logit first. Against oracle/ends.py in float64, with the tolerances of
test_gpu_logits.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from test_gpu_logits import _check_distill, _logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


# several CTAs a row, one of 256 threads, of 128, of 64
@pytest.mark.parametrize("N,V", [(9, 90001), (9, 700), (1500, 20000), (310, 5000), (2500, 2000)])
@pytest.mark.parametrize("K,copies", [(5, 5), (40, 4), (300, 3), (300, 60), (1024, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_listed_many_times(N, V, K, copies, dtype):
    rng = np.random.default_rng(K + copies)
    z = _logits(rng, N, V, dtype)
    apart = K // copies
    idx = np.stack([rng.choice(min(V, 700), apart, replace=False) for _ in range(N)]).astype(np.int32)
    idx = np.concatenate([idx] * copies + [np.full((N, K - apart * copies), -1, dtype=np.int32)], axis=1)
    idx[1] = idx[1][rng.permutation(K)]  # in no order
    labels = torch.from_numpy(idx[:, K // 2].copy()).cuda()
    idx = torch.from_numpy(idx).cuda()
    val = torch.from_numpy(rng.normal(0, 1, (N, K)).astype(np.float32)).cuda()
    rest = torch.zeros(N, device="cuda")
    few = torch.tensor([0, 1, 4, N - 1], device="cuda")
    for tau, kd, ce in ((1.5, 0.5, 0.5), (1.0, 1.0, 0.0)):
        op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=tau, kd_weight=kd, ce_weight=ce)
        loss, dz = op.forward_backward(z, idx, val, rest=rest, labels=labels if ce else None)
        tw.raise_if_device_error(op.status)
        assert torch.isfinite(loss).all() and torch.isfinite(dz).all()
        _check_distill(loss[few], dz[few], z[few], idx[few], val[few], rest[few], labels[few] if ce else None, tau, kd, ce)
