"""Where the orthogonalised update's precision comes from, on the CPU: a model of the products'
roundings (fp16 operands, X as hi + lo, fp32 sums) is as precise as the header says, and is not
once one of the choices is taken out. test_gpu_ortho_ranks.py holds the kernels to the same
bounds."""
import numpy as np
import pytest

from oracle import updates

A, B, C = updates.COEFFICIENTS
EPS = 2.0 ** -12.24  # an fp16 rounding in the quadratic mean over mantissas


def _f16(x):
    return x.astype(np.float16).astype(np.float32)


def _model(u, steps, t_one=lambda s, n: s >= 3 and s + 1 == n, lo=True, diagonal=True, operands=_f16):
    """`steps` of X <- q0 X + X (q1 E + c E^2), E = X^T X - t, as tw_ortho.cu has them."""
    k = min(14, max(0, round(0.5 * np.log2(u.size))))
    x = (u / np.linalg.norm(u)).astype(np.float32) * np.float32(2.0 ** k)
    eye = np.eye(u.shape[1], dtype=np.float32)
    for s in range(steps):
        hi = _f16(x)
        x = hi + _f16(x - hi) if lo else hi
        t = 1.0 if t_one(s, steps) else 0.0
        q0, q1, operand = np.float32(A + B * t + C * t * t), np.float32(B + 2 * C * t), operands(hi)
        e = operands((operand.T @ operand) * np.float32(2.0 ** (12 - 2 * k)) - np.float32(2.0 ** 12 * t) * eye)
        b = e * (q1 / 4) + (e @ e) * np.float32(C * 2.0 ** -14)
        lost = np.diag(b - operands(b)) if diagonal else 0.0
        x = x * (q0 + lost * np.float32(2.0 ** -10)) + (operand @ operands(b)) * np.float32(2.0 ** -10)
    return x * np.float32(2.0 ** -k)


def _error(u, steps=5, **kw):
    want = updates.newton_schulz(u, steps)
    return np.linalg.norm(_model(u, steps, **kw) - want) / np.linalg.norm(want)


def _tol(steps):  # derived in test_gpu_ortho_ranks.py
    return 5.05 * EPS * max(1, steps - 2) ** 0.5 + 2.0 ** -23 * 3.4445 ** steps


def _rank(m, n, r):
    rng = np.random.default_rng(m + r)
    return rng.normal(size=(m, r)) @ rng.normal(size=(r, n))


def _steep(spread):
    rng = np.random.default_rng(6)
    u, v = np.linalg.qr(rng.normal(size=(400, 160)))[0], np.linalg.qr(rng.normal(size=(160, 160)))[0]
    return (u * np.arange(1, 161) ** -spread) @ v


@pytest.mark.parametrize("steps", [5, 6, 8])
@pytest.mark.parametrize("r", [1, 8, 40, 128])
def test_any_rank(r, steps):
    u = _rank(300, 128, r)
    assert _error(u, steps) <= _tol(steps)
    if r < 128:  # t = 1 as soon as the largest values are near 1: not where others are 0
        assert _error(u, steps, t_one=lambda s, n: s >= 3) > _tol(steps)


@pytest.mark.parametrize("spread", [1.0, 1.5, 2.0])
def test_steep_spectra(spread):
    assert _error(_steep(spread)) <= _tol(5)


def test_what_each_choice_is_for():
    assert _error(_steep(1.5), lo=False) > 2 * _tol(5)                      # X in 11 bits
    bf16 = lambda x: (x.astype(np.float32).view(np.uint32) + 0x8000 & 0xFFFF0000).view(np.float32)  # noqa: E731
    assert _error(_rank(300, 128, 128), operands=bf16) > 2 * _tol(5)        # operands of 8 bits
    # full rank: the last step's t, and the diagonal in fp32
    full = [_rank(300, 128, 128) + seed for seed in range(3)]
    as_it_is = max(_error(u) for u in full)
    assert min(_error(u, diagonal=False) for u in full) > as_it_is
    assert min(_error(u, diagonal=False, t_one=lambda s, n: False) for u in full) > 1.3 * as_it_is
