"""Orthogonalised updates of matrices of few singular values, of full rank and of steep spectra,
over several numbers of steps, against oracle/updates.py in float64; results in fp32, so that
the products' roundings alone are seen.

Tolerance, in the Frobenius norm, from the arithmetic. A rounding to fp16 is at most 2^-11 of the
value and eps = 2^-11 sqrt(3 / (8 ln 2) / 3) = 2^-12.24 in the quadratic mean over mantissas.
With the usual coefficients a step takes in, of X's norm and singular values s^(1/2) up to 1.2:
X's hi in the product with B, |B| = |b s + c s^2| <= 2.81: 2.81 eps; B's own, the same; E's,
|b s + 2 c s^2| <= 1.4: 1.4 eps; hi in the gram, twice that: 2.8 eps. Together, as independent
ones, 5.05 eps. The first steps multiply X by up to 3.44, which makes theirs small; of `steps` all
but two count. Where U's singular value is 0 X keeps roundings of 2^-23 (hi + lo), which each
step multiplies by 3.44.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import updates  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -12.24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _tol(steps, eps=EPS):
    return 5.05 * eps * max(1, steps - 2) ** 0.5 + 2.0 ** -23 * 3.4445 ** steps


def _error(op, u):
    """|got - want| / |want| of one matrix."""
    g = torch.from_numpy(u.astype(np.float32)).cuda()
    got = op(g).double().cpu().numpy()
    want = updates.newton_schulz(g.double().cpu().numpy(), op.steps)
    assert np.isfinite(got).all()
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def _op(m, n, steps):
    return tw.Orthogonalize(m, n, steps=steps, momentum=0.0, dtype=torch.float32)


def _rank(rng, m, n, r):
    return rng.normal(size=(m, r)) @ rng.normal(size=(r, n))


@pytest.mark.parametrize("steps", [4, 5, 6, 8])
@pytest.mark.parametrize("m,n,r", [(500, 200, 1), (500, 200, 8), (200, 500, 8), (500, 200, 60), (600, 512, 77), (70, 90, 3),
                                   (500, 200, 200), (300, 700, 300), (64, 64, 64)])
def test_ranks_and_steps(m, n, r, steps):
    err = _error(_op(m, n, steps), _rank(np.random.default_rng(m + r), m, n, r))
    assert err <= _tol(steps), f"{err:.3g}"


@pytest.mark.parametrize("spread", [1.0, 1.5, 2.0])
def test_steep_spectra(spread):
    """Singular values over two to five decades, most of them still rising after five steps: X in
    11 bits alone, or operands of 8 bits, are 4e-3 to 1e-2 off."""
    rng = np.random.default_rng(6)
    u, v = np.linalg.qr(rng.normal(size=(500, 200)))[0], np.linalg.qr(rng.normal(size=(200, 200)))[0]
    err = _error(_op(500, 200, 5), (u * np.arange(1, 201) ** -spread) @ v)
    assert err <= _tol(5), f"{err:.3g}"


@pytest.mark.parametrize("m,n", [(1, 1), (7, 1), (1, 9), (3, 2), (4, 64), (8, 8)])
def test_few_rows_or_columns(m, n):
    """One rounding is then the whole error: half a step, 2^-11, in place of the mean; and at its
    largest a step moves a relative error by |s p'(s) / p(s)| = 5 (singular value 1.2)."""
    op = _op(m, n, 5)
    errs = [_error(op, np.random.default_rng(seed).normal(size=(m, n))) for seed in range(60)]
    assert np.median(errs) <= _tol(5, 2.0 ** -11), f"{np.median(errs):.3g}"
    assert max(errs) <= 5 * _tol(5, 2.0 ** -11), f"{max(errs):.3g}"
