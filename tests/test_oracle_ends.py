"""Pins of oracle/ends.py (float64 definitions of layer norm, the distillation loss and
token log probabilities): closed forms, central differences and torch autograd in
float64, written apart from the oracle."""
import math

import numpy as np
import pytest

from oracle import ends

torch = pytest.importorskip("torch")


def _central(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        p, m = x.copy(), x.copy()
        p[i] += h
        m[i] -= h
        g[i] = (f(p) - f(m)) / (2 * h)
    return g


# a central difference of a smooth O(1) function in fp64 at h = 1e-5: truncation ~h^2,
# rounding ~eps / h: both about 1e-10
FD = dict(rtol=1e-6, atol=1e-8)


def test_layer_norm_closed_forms():
    y, mean, rstd = ends.layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), eps=0.25)
    np.testing.assert_allclose(mean, [2, 5])
    np.testing.assert_allclose(rstd, [1 / math.sqrt(1.25), 2.0])
    np.testing.assert_allclose(y, [[-1 / math.sqrt(1.25), 1 / math.sqrt(1.25)], [0, 0]])
    y, _, _ = ends.layer_norm(np.array([[7.0, 7.0, 7.0]]), np.array([2.0, 3, 4]), np.array([1.0, 0, -1]))
    np.testing.assert_allclose(y, [[1, 0, -1]])


def test_layer_norm_matches_torch():
    rng = np.random.default_rng(0)
    s, w, b = rng.normal(3, 2, (5, 11)), rng.normal(size=11), rng.normal(size=11)
    dy, dres = rng.normal(size=(5, 11)), rng.normal(size=(5, 11))
    ts, tw, tb = (torch.tensor(v, requires_grad=True) for v in (s, w, b))
    ty = torch.nn.functional.layer_norm(ts, (11,), tw, tb, 1e-5)
    np.testing.assert_allclose(ends.layer_norm(s, w, b)[0], ty.detach().numpy(), rtol=1e-12, atol=1e-13)
    ((ty * torch.tensor(dy)).sum() + (ts * torch.tensor(dres)).sum()).backward()
    for got, ref in zip(ends.layer_norm_grad(dy, s, w, dres=dres), (ts.grad, tw.grad, tb.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-10, atol=1e-12)


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy = rng.normal(size=(3, 6)), rng.normal(size=6), rng.normal(size=(3, 6))
    dx, dw, _ = ends.layer_norm_grad(dy, s, w)
    np.testing.assert_allclose(dx, _central(lambda v: (dy * ends.layer_norm(v, w)[0]).sum(), s), **FD)
    np.testing.assert_allclose(dw, _central(lambda v: (dy * ends.layer_norm(s, v)[0]).sum(), w), **FD)


def _case(seed, N=4, V=9, K=3, dup=False):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, (N, V))
    idx = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    idx[1, 1:] = -1
    if dup:
        idx[2, 2] = idx[2, 0]
    return dict(z=z, idx=idx, val=rng.normal(0, 2, (N, K)), rest=rng.normal(size=N), labels=np.array([2, -1, 0, 5][:N]))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tau,kd_w,ce_w", [(1.0, 1.0, 0.0), (2.0, 0.7, 0.3), (0.5, 0.0, 1.0)])
@pytest.mark.parametrize("dup", [False, True])
def test_distill_gradient_against_differences(rest, tau, kd_w, ce_w, dup):
    c = _case(3, dup=dup)
    args = dict(idx=c["idx"], val=c["val"], rest=c["rest"] if rest else None, labels=c["labels"], temperature=tau,
                kd_weight=kd_w, ce_weight=ce_w)
    up = np.array([1.0, 2.0, -0.5, 3.0])
    _, dz = ends.distill(c["z"], dloss=up, scale=0.25, **args)
    num = _central(lambda v: (ends.distill(v, **args)[0] * up).sum() * 0.25, c["z"])
    np.testing.assert_allclose(dz, num, **FD)


def test_distill_full_list_is_kullback_leibler():
    rng = np.random.default_rng(4)
    z, t, tau = rng.normal(size=(3, 5)), rng.normal(size=(3, 5)), 1.7
    idx = np.tile(np.arange(5, dtype=np.int32)[::-1], (3, 1))
    loss, _ = ends.distill(z, idx, t[:, ::-1], temperature=tau)
    lp, lq = torch.log_softmax(torch.tensor(t) / tau, 1), torch.log_softmax(torch.tensor(z) / tau, 1)
    np.testing.assert_allclose(loss, ((lp.exp() * (lp - lq)).sum(1) * tau ** 2).numpy(), rtol=1e-12)


def test_distill_rest_bucket_is_the_teachers_tail():
    """With the rest given, P is the teacher's own distribution, and a student equal to the
    teacher has loss 0 and gradient 0."""
    rng = np.random.default_rng(5)
    t = rng.normal(size=(2, 8))
    idx = np.argsort(-t, axis=1)[:, :3].astype(np.int32)
    val = np.take_along_axis(t, idx, 1)
    rest = np.array([np.log(sum(math.exp(t[n, v]) for v in range(8) if v not in idx[n])) for n in range(2)])
    loss, dz = ends.distill(t, idx, val, rest=rest)
    np.testing.assert_allclose(loss, 0, atol=1e-12)
    np.testing.assert_allclose(dz, 0, atol=1e-12)
    # without it the renormalised list differs from the student's mass on it
    assert (ends.distill(t, idx, val)[0] > 1e-3).all()


def test_distill_cross_entropy_and_empty_rows():
    z = np.array([[0.0, math.log(3.0)], [1.0, 2.0], [-np.inf, -np.inf], [np.nan, 0.0]])
    loss, dz = ends.distill(z, labels=np.array([1, -1, 0, -1]), kd_weight=0.0, ce_weight=1.0)
    np.testing.assert_allclose(loss, [-math.log(0.75), 0, np.inf, 0])
    np.testing.assert_allclose(dz, [[0.25, -0.25], [0, 0], [0, 0], [0, 0]])


def test_token_logprobs_closed_form_ties_and_masks():
    z = np.array([[0.0, 0.0, math.log(2.0), -0.0], [-np.inf, 1.0, -np.inf, -np.inf], [-np.inf] * 4, [0, np.inf, 0, 0]])
    lp, ent, idx, top = ends.token_logprobs(z, np.array([[2, -1]] * 4), top_k=3)
    np.testing.assert_array_equal(idx, [[2, 0, 1], [1, -1, -1], [-1, -1, -1], [-1, -1, -1]])
    np.testing.assert_allclose(lp[:, 0], [math.log(0.4), -np.inf, -np.inf, np.nan])
    np.testing.assert_array_equal(lp[:, 1], 0)
    np.testing.assert_allclose(ent, [-(0.4 * math.log(0.4) + 0.6 * math.log(0.2)), 0, 0, np.nan], atol=1e-12)
    np.testing.assert_allclose(top[0], np.log([0.4, 0.2, 0.2]))
    np.testing.assert_array_equal(top[1], [0, -np.inf, -np.inf])
