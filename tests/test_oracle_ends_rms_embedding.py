"""Pins of the RMS norm, e4m3 and embedding parts of oracle/ends.py: closed forms, finite
differences, the format's table, and planted mistakes."""
import numpy as np
import pytest

from oracle import ends

RNG = np.random.default_rng(17)


def test_rms_norm_by_hand():
    y, rstd = ends.rms_norm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([2.0, 1.0]), eps=0.0 + 1e-300)
    assert np.allclose(rstd[0], 1 / np.sqrt(12.5)) and np.allclose(y[0], [6 / np.sqrt(12.5), 4 / np.sqrt(12.5)])
    assert not y[1].any()


def test_rms_norm_is_layer_norm_of_a_centred_row():
    s = RNG.normal(size=(5, 12))
    s -= s.mean(axis=1, keepdims=True)
    assert np.abs(ends.rms_norm(s, eps=1e-5)[0] - ends.layer_norm(s, eps=1e-5)[0]).max() < 1e-13


def _loss(dy, s, w, dres):
    return (dy * ends.rms_norm(s, w, 1e-3)[0]).sum() + (dres * s).sum()


def test_rms_norm_grad_by_differences():
    s, w, dy, dres = RNG.normal(size=(3, 7)), RNG.normal(size=7), RNG.normal(size=(3, 7)), RNG.normal(size=(3, 7))
    dx, dw = ends.rms_norm_grad(dy, s, w, 1e-3, dres)
    h = 1e-6
    for t, c in np.ndindex(3, 7):
        e = np.zeros((3, 7))
        e[t, c] = h
        assert abs((_loss(dy, s + e, w, dres) - _loss(dy, s - e, w, dres)) / (2 * h) - dx[t, c]) < 1e-7
    for c in range(7):
        e = np.zeros(7)
        e[c] = h
        assert abs((_loss(dy, s, w + e, dres) - _loss(dy, s, w - e, dres)) / (2 * h) - dw[c]) < 1e-7


def test_e4m3_table_and_rounding():
    torch = pytest.importorskip("torch")
    grid = ends.e4m3_values()
    assert grid[-1] == 448 and grid[1] == 2.0 ** -9 and (np.diff(grid) > 0).all()
    table = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (table == grid).all()
    v = np.concatenate([RNG.normal(size=2000) * 100, RNG.normal(size=500) * 2.0 ** -8, (grid[1:] + grid[:-1]) / 2, -grid, [0.0, 448.0]])
    v = v.astype(np.float32)
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert (ends.to_e4m3(v.astype(np.float64)) == want).all()


def test_scales():
    y = np.array([[1.0, -896.0, 4.0], [0.0, 0.0, 0.0]])
    assert ends.fp8_scales(y).tolist() == [[2.0], [2.0 ** -126]]
    assert ends.fp8_scales(y, 2).tolist() == [[2.0, 4.0 / 448.0], [2.0 ** -126, 2.0 ** -126]]


def test_embedding_grad_is_the_transpose_of_the_forward():
    tokens = np.array([3, -1, 0, 3, 3, 4])
    w, dy = RNG.normal(size=(6, 5)), RNG.normal(size=(6, 5))
    assert np.isclose((dy * ends.embedding(tokens, w, 1.5)).sum(), (ends.embedding_grad(dy, tokens, 6, 1.5) * w).sum())
    assert not ends.embedding(tokens, w)[1].any()
    one_hot = np.zeros((6, 6))
    one_hot[np.arange(6)[tokens >= 0], tokens[tokens >= 0]] = 1
    assert np.abs(ends.embedding_grad(dy, tokens, 6) - one_hot.T @ dy).max() < 1e-14


@pytest.mark.parametrize("wrong", ["mean", "no_c2", "wrong_row"])
def test_planted_mistakes_fail_the_pins(wrong):
    s, w, dy = RNG.normal(1.0, 1.0, size=(3, 7)), RNG.normal(size=7), RNG.normal(size=(3, 7))
    dx, _ = ends.rms_norm_grad(dy, s, w, 1e-3)
    bad = {"mean": ends.layer_norm_grad(dy, s, w, 1e-3)[0],
           "no_c2": ends.rms_norm(s, eps=1e-3)[1][:, None] * dy * w,
           "wrong_row": ends.rms_norm_grad(dy[::-1], s, w, 1e-3)[0]}[wrong]
    assert np.abs(bad - dx).max() > 1e-3
