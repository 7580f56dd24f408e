"""The distillation where the unlisted tokens lie far below the listed ones: their mass under
the student is less than fp32's smallest number, while its logarithm, and the term
P_rest q / q_rest of the gradient (it sums to P_rest), are ordinary numbers.

Against oracle/ends.py in float64. Tolerances: test_gpu_logits.py's for the gradient; the loss,
whose size is the gap's, to 4 R relative beside the terms of ordinary size.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import ends  # noqa: E402
from test_gpu_logits import R, _check_distill, _f64  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _case(N, V, K, dtype, gap, masked):
    """Listed tokens `gap` above the unlisted ones, of which some are -inf where `masked`; labels
    listed, unlisted and none."""
    rng = np.random.default_rng(V + K)
    z = rng.normal(0, 1.5, (N, V)).astype(np.float32)
    idx = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    lab = np.where(np.arange(N) % 3 == 0, idx[:, 1], rng.integers(0, V, N)).astype(np.int32)
    lab[np.arange(N) % 5 == 4] = -1
    hide = rng.random((N, V)) < 0.3 if masked else np.zeros((N, V), dtype=bool)
    np.put_along_axis(hide, idx, False, 1)
    hide[np.nonzero(lab >= 0)[0], lab[lab >= 0]] = False
    z[hide] = -np.inf
    np.put_along_axis(z, idx, np.take_along_axis(z, idx, 1) + np.float32(gap), 1)
    val = rng.normal(1, 1, (N, K)).astype(np.float32)
    rest = rng.normal(0, 1, N).astype(np.float32)
    rest[1] = -np.inf  # one row without a rest
    z = torch.from_numpy(z).to(dtype).cuda()
    return z, *(torch.from_numpy(t).cuda() for t in (idx, val, rest, lab))


def _check(op, args, few, tau, kd, ce, dloss, scale):
    z, idx, val, rest, lab = args
    lab = lab if ce else None
    loss, dz = op.forward_backward(z, idx, val, rest=rest, labels=lab, dloss=dloss, scale=scale)
    tw.raise_if_device_error(op.status)
    one = lambda t: None if t is None else t[few]  # noqa: E731
    _check_distill(loss[few], dz[few], z[few], idx[few], val[few], rest[few], one(lab), tau, kd, ce, one(dloss), scale)
    n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    with np.errstate(over="ignore"):
        want = ends.distill(_f64(z[few]), n(idx[few]), _f64(val[few]), _f64(rest[few]), n(one(lab)), tau, kd, ce)[0]
    assert np.isfinite(want).all()
    got = _f64(loss[few])
    assert (np.abs(got - want) <= 4 * R * (np.abs(want) + 20 * (1 + tau * tau))).all(), (got, want)
    # the loss alone, which long rows take another way
    assert (torch.abs(op.forward(z, idx, val, rest=rest, labels=lab)[few].double().cpu() - torch.from_numpy(want))
            <= 4 * R * (torch.from_numpy(np.abs(want)) + 20 * (1 + tau * tau))).all()


# several CTAs a row, one of 256 threads, of 128, of 64
SIZES = [(7, 1000, 5), (7, 90001, 40), (170, 18001, 40), (310, 2000, 40), (2500, 515, 6)]


@pytest.mark.parametrize("N,V,K", SIZES)
@pytest.mark.parametrize("gap", [30.0, 80.0, 86.0, 88.0, 92.0, 100.0, 130.0, 1000.0])
@pytest.mark.parametrize("dtype,scale", [(F32, 1.0), (BF16, 1.0), (F16, 2.0 ** 15)])
def test_listed_tokens_far_above_the_rest(N, V, K, gap, dtype, scale):
    args = _case(N, V, K, dtype, gap, masked=True)
    few = torch.tensor([0, 1, 2, 3, 4, N // 2, N - 1], device="cuda")
    for tau, kd, ce in ((1.0, 1.0, 0.0), (1.0, 0.5, 0.5), (0.1, 0.7, 0.3), (2.0, 0.7, 0.3)):
        op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=tau, kd_weight=kd, ce_weight=ce)
        _check(op, args, few, tau, kd, ce, None, scale)


@pytest.mark.parametrize("N,V,K", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tau", [1.0, 0.1, 2.0])
def test_unlisted_tokens_at_the_lowest_value(N, V, K, dtype, tau):
    """A mask of the type's lowest finite value is a number: the rest is uniform over it."""
    z, idx, val, rest, lab = _case(N, V, K, dtype, 0.0, masked=False)
    keep = torch.zeros(z.shape, dtype=torch.bool, device="cuda").scatter_(1, idx.long(), True)
    keep[torch.nonzero(lab >= 0)[:, 0], lab[lab >= 0].long()] = True
    z = torch.where(keep, z, torch.full_like(z, torch.finfo(dtype).min))
    lab = torch.where(torch.arange(N, device="cuda") % 3 == 0, idx[:, 1], -1).to(torch.int32)  # nothing else unmasked
    z = torch.where(torch.zeros_like(keep).scatter_(1, idx.long(), True), z, torch.full_like(z, torch.finfo(dtype).min))
    few = torch.tensor([0, 1, 2, 3, 4, N // 2, N - 1], device="cuda")
    for kd, ce in ((0.3, 0.0), (0.3, 0.5)):
        op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=tau, kd_weight=kd, ce_weight=ce)
        _check(op, (z, idx, val, rest, lab), few, tau, kd, ce, None, 1.0)


@pytest.mark.parametrize("N,V,K", SIZES)
def test_rows_far_apart_with_the_rest_above(N, V, K):
    """The same gap the other way: the listed tokens far below, and the rest's mass is all."""
    args = _case(N, V, K, F32, -150.0, masked=True)
    few = torch.tensor([0, 1, 2, 3, 4, N // 2, N - 1], device="cuda")
    for tau, kd, ce in ((1.0, 1.0, 0.0), (2.0, 0.7, 0.3)):
        op = tw.DistillLoss(N, V, K, dtype=F32, temperature=tau, kd_weight=kd, ce_weight=ce)
        _check(op, args, few, tau, kd, ce, None, 1.0)
