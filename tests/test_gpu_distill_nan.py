"""A NaN in a row makes its loss and gradient NaN wherever it lies: here in a stretch of -inf
that fills the first loads of every thread that meets it, with numbers only after it.

Against oracle/ends.py in float64, with the tolerances of test_gpu_logits.py for the rows
without a NaN.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from test_gpu_logits import _check_distill, _logits, _teacher  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _rows_with_nan(N, V, dtype, period, share):
    """Logits whose rows 1 to 4 are -inf over the first `share` of every `period` columns, rows
    2 to 4 with a NaN there, and the same logits without the NaNs."""
    rng = np.random.default_rng(V)
    z = _logits(rng, N, V, dtype, pad=(8 - V) % 8)
    idx, val = _teacher(rng, z, 9, ragged=False)
    z[1:5, (torch.arange(V, device="cuda") % period) < int(share * period)] = -INF
    clean = z.clone()
    for row, at in ((2, 0), (3, 611), (4, 1500)):
        z[row, at] = float("nan")
    # listed: some masked, some not (numbers must be left where the teacher has mass)
    idx[1:5, 4:] = torch.arange(period - 5, period, device="cuda", dtype=torch.int32)
    idx[1:5, :4] = torch.arange(20, 24, device="cuda", dtype=torch.int32)
    val[1:5, :4] = -INF
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    labels[1:5] = period - 7
    return z, clean, idx, val, labels


# sizes whose kernels are: a row over several CTAs, over one of 256 threads, one CTA of 128
# and of 64 threads a row. The stretch is longer than a thread's first four vectors.
@pytest.mark.parametrize("N,V,period,share", [(6, 90000, 11250, 0.85), (170, 18000, 18000, 0.6), (310, 13000, 13000, 0.6),
                                              (2500, 6000, 6000, 0.6)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tau,kd,ce", [(1.0, 1.0, 0.0), (1.0, 0.5, 0.5), (1.5, 0.5, 0.5), (2.0, 0.5, 0.5), (4.0, 0.5, 0.5),
                                       (2.0, 0.0, 1.0)])
def test_nan_in_a_masked_stretch(N, V, period, share, dtype, tau, kd, ce):
    z, clean, idx, val, labels = _rows_with_nan(N, V, dtype, period, share)
    op = tw.DistillLoss(N, V, 9, dtype=dtype, temperature=tau, kd_weight=kd, ce_weight=ce)
    lab = labels if ce else None
    loss, dz = op.forward_backward(z, idx, val, labels=lab)
    assert torch.isnan(loss[2:5]).all() and torch.isnan(dz[2:5]).all()
    few = torch.tensor([0, 1, 2, 3, 4, 5, N - 1], device="cuda")
    _check_distill(loss[few], dz[few], z[few], idx[few], val[few], None, None if lab is None else lab[few], tau, kd, ce)
    others = torch.ones(N, dtype=torch.bool, device="cuda")
    others[2:5] = False
    loss, dz = loss.clone(), dz.clone()
    l2, d2 = op.forward_backward(clean, idx, val, labels=lab)
    assert torch.isfinite(l2).all() and torch.isfinite(d2).all()
    assert torch.equal(loss[others], l2[others]) and torch.equal(dz[others], d2[others])


@pytest.mark.parametrize("dtype,N,V", [(F32, 170, 60000), (BF16, 1300, 32000), (F16, 2500, 6000)])
@pytest.mark.parametrize("tau,ce", [(1.0, 0.0), (1.5, 0.5), (2.0, 0.5)])
def test_nan_in_a_masked_stretch_of_the_loss_alone(dtype, N, V, tau, ce):
    z, clean, idx, val, labels = _rows_with_nan(N, V, dtype, V, 0.6)
    op = tw.DistillLoss(N, V, 9, dtype=dtype, temperature=tau, kd_weight=0.5, ce_weight=ce, grad=False)
    lab = labels if ce else None
    loss = op.forward(z, idx, val, labels=lab).clone()
    assert torch.isnan(loss[2:5]).all()
    l2 = op.forward(clean, idx, val, labels=lab)
    assert torch.isfinite(l2).all()
    assert torch.equal(loss[:2], l2[:2]) and torch.equal(loss[5:], l2[5:])
