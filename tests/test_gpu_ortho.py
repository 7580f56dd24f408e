"""GPU parity of the orthogonalised updates against oracle/updates.py in float64.

Tolerances, from the arithmetic. Three operands a step are rounded to fp16, by at most half
a step, 2^-11 of the value, and by 2^-12 or less in the quadratic mean; so 15 in five steps.
The step's polynomial moves relative errors by a factor of about 1 in the mean
(|s p'(s) / p(s)| <= 1.4 below the largest singular values, smaller near 1). Added linearly
that is 15 * 2^-11 = 7.4e-3 of the result's 2-norm for a matrix of few singular values, where
one rounding is the whole error, and 15 * 2^-12 = 3.7e-3 from 64 on, where the roundings of a
product are many and independent and the 2-norm sees their quadratic mean. A rounding of the
result to its type (u) comes on top. Momentum is two fp32 operations: 2^-23 of |mu M| + |G|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import updates  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
ROUNDINGS = 15


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _grad(rng, m, n, dtype=F32, scale=1.0):
    """Rows and columns of unlike sizes, and a few shared directions."""
    rows, cols = np.exp(rng.normal(size=(m, 1))), (1.0 + rng.permutation(n)) ** -0.5
    g = rng.normal(size=(m, n)) * rows * cols
    k = min(4, m, n)
    g += 0.3 * (rng.normal(size=(m, k)) * rows) @ (rng.normal(size=(k, n)) * cols)
    return torch.from_numpy((g * scale).astype(np.float32)).to(dtype).cuda()


def _tol(m, n, roundings=ROUNDINGS):
    return roundings * (2.0 ** -12 if min(m, n) >= 64 else 2.0 ** -11)


def _check(got, want, dtype, roundings=ROUNDINGS):
    got, tol = _f64(got), _tol(*got.shape, roundings)
    assert np.isfinite(got).all()
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= (tol + U[dtype]) * norm, f"{err / norm:.3g} off in the 2-norm"


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 2), (64, 64), (65, 63), (255, 256), (257, 255), (128, 1027), (704, 256), (300, 700),
          (520, 513), (2000, 130), (33, 4100), (1024, 1024)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("gdtype,dtype,momentum", [(F32, BF16, 0.95), (BF16, BF16, 0.0), (F16, F32, 0.9), (F32, F16, 0.0)])
def test_matches_oracle(m, n, gdtype, dtype, momentum):
    rng = np.random.default_rng(m * 31 + n)
    g = _grad(rng, m, n, gdtype)
    buf = _grad(rng, m, n) if momentum else None
    was = None if buf is None else _f64(buf)
    op = tw.Orthogonalize(m, n, dtype=dtype, grad_dtype=gdtype, momentum=momentum)
    out = op(g, buf, scale=1.5)
    torch.cuda.synchronize()
    tw.raise_if_device_error(op.status)
    u = _f64(g)
    if momentum:
        new, u = updates.momentum(u, was, momentum)
        assert (np.abs(_f64(buf) - new) <= 2.0 ** -23 * (np.abs(momentum * was) + np.abs(_f64(g)))).all()
        u = _f64(g) + momentum * _f64(buf)
    _check(out, 1.5 * updates.newton_schulz(u), dtype)


@pytest.mark.parametrize("count", [2, 3, 8])
@pytest.mark.parametrize("m,n", [(300, 520), (520, 300), (64, 64)])
def test_several_at_once_are_each_alone(m, n, count):
    rng = np.random.default_rng(count)
    gs, bufs = [_grad(rng, m, n, scale=10.0 ** i) for i in range(count)], [_grad(rng, m, n) for _ in range(count)]
    copies = [b.clone() for b in bufs]
    op = tw.Orthogonalize(m, n, count=count)
    outs = [o.clone() for o in op(gs, bufs)]
    for g, b, c, o in zip(gs, bufs, copies, outs):
        one = tw.Orthogonalize(m, n)(g, c)
        assert torch.equal(b, c)
        _check(o, _f64(one), BF16)
        _check(o, updates.newton_schulz(_f64(g) + 0.95 * _f64(b)), BF16)
    # fewer than the object was made for
    few = op(gs[:1], [bufs[0].clone()])
    assert len(few) == 1


def test_the_same_call_gives_the_same_bits():
    rng = np.random.default_rng(3)
    g = _grad(rng, 1500, 700)
    op = tw.Orthogonalize(1500, 700, momentum=0.0)
    first = op(g).clone()
    for _ in range(5):
        assert torch.equal(op(g), first)
    op.ws.fill_(255)  # whatever the workspace holds
    assert torch.equal(op(g), first)


@pytest.mark.parametrize("gdtype,scale", [(F32, 1e-38), (F32, 1e-30), (F32, 1e30), (F32, 3e37), (BF16, 1e-36), (F16, 1e-6)])
def test_norms_far_from_one(gdtype, scale):
    rng = np.random.default_rng(9)
    g = torch.from_numpy(rng.normal(size=(130, 70)).astype(np.float64) * scale).to(gdtype).cuda()
    op = tw.Orthogonalize(130, 70, grad_dtype=gdtype, momentum=0.0)
    _check(op(g), updates.newton_schulz(_f64(g)), BF16)


def test_zero_nan_and_infinity():
    op = tw.Orthogonalize(80, 90, momentum=0.0)
    assert not op(torch.zeros(80, 90, device="cuda")).any()
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = _grad(np.random.default_rng(1), 80, 90)
        g[79, 3] = bad
        assert torch.isnan(op(g)).all()
    # and the next call is clean again
    g = _grad(np.random.default_rng(2), 80, 90)
    _check(op(g), updates.newton_schulz(_f64(g)), BF16)


def test_rank_one_and_dead_rows():
    rng = np.random.default_rng(4)
    g = torch.zeros(600, 300, device="cuda")
    g[100] = torch.from_numpy(rng.normal(size=300).astype(np.float32)).cuda()
    op = tw.Orthogonalize(600, 300, momentum=0.0)
    _check(op(g), updates.newton_schulz(_f64(g)), BF16)
    g = _grad(rng, 600, 300)
    g[::2] = 0
    got = op(g)
    assert not got[::2].any()
    _check(got, updates.newton_schulz(_f64(g)), BF16)


@pytest.mark.parametrize("spread", [0.5, 1.0, 1.5])
def test_spectra_over_decades(spread):
    rng = np.random.default_rng(6)
    u, v = np.linalg.qr(rng.normal(size=(500, 200)))[0], np.linalg.qr(rng.normal(size=(200, 200)))[0]
    g = torch.from_numpy(((u * np.arange(1, 201) ** -spread) @ v).astype(np.float32)).cuda()
    _check(tw.Orthogonalize(500, 200, momentum=0.0)(g), updates.newton_schulz(_f64(g)), BF16)


@pytest.mark.parametrize("steps,coef", [(1, updates.COEFFICIENTS), (2, updates.COEFFICIENTS), (8, updates.COEFFICIENTS),
                                        (3, [(4.0, -6.0, 2.5), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375)])])
def test_steps_and_coefficients(steps, coef):
    rng = np.random.default_rng(8)
    g = _grad(rng, 210, 150)
    op = tw.Orthogonalize(210, 150, steps=steps, coefficients=coef, momentum=0.0, dtype=F32)
    _check(op(g), updates.newton_schulz(_f64(g), steps, coef), F32, roundings=max(5, 3 * steps))


@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_forms(nesterov):
    rng = np.random.default_rng(10)
    g, b = _grad(rng, 90, 140), _grad(rng, 90, 140)
    _, u = updates.momentum(_f64(g), _f64(b), 0.7, nesterov)
    op = tw.Orthogonalize(90, 140, momentum=0.7, nesterov=nesterov)
    _check(op(g, b), updates.newton_schulz(u), BF16)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,n", [(200, 300), (300, 200), (301, 77)])
def test_weights_updated_in_place_between_others(m, n, dtype):
    """Strided gradients, buffers and weights with guards around the rows."""
    rng = np.random.default_rng(m)

    def inside(t, off, pad, fill):
        big = torch.full((m + 2, off + n + pad), fill, dtype=t.dtype, device="cuda")
        big[1:m + 1, off:off + n] = t
        return big, big[1:m + 1, off:off + n]

    g0, b0 = _grad(rng, m, n), _grad(rng, m, n)
    w0 = torch.from_numpy(rng.normal(size=(m, n)).astype(np.float32) * 0.05).to(dtype).cuda()
    (_, g), (bb, b), (wb, w) = inside(g0, 3, 2, float("nan")), inside(b0, 1, 4, 7.0), inside(w0, 5, 0, 9.0)
    op = tw.Orthogonalize(m, n, dtype=dtype)
    res = op(g, b, out=w, scale=-0.1, beta=0.9)
    assert res is w or res.data_ptr() == w.data_ptr()
    new, u = updates.momentum(_f64(g0), _f64(b0), 0.95)
    x = updates.newton_schulz(u)
    want = 0.9 * _f64(w0) - 0.1 * x
    got = _f64(w)
    assert np.linalg.norm(got - want) <= U[dtype] * np.linalg.norm(want) + _tol(m, n) * 0.1 * np.linalg.norm(x)
    assert (wb[0] == 9).all() and (wb[-1] == 9).all() and (wb[:, :5] == 9).all()
    assert (bb[0] == 7).all() and (bb[-1] == 7).all() and (bb[:, :1] == 7).all() and (bb[:, 1 + n:] == 7).all()


def test_result_may_replace_the_gradient():
    g = _grad(np.random.default_rng(12), 333, 257, BF16)
    want = updates.newton_schulz(_f64(g))
    op = tw.Orthogonalize(333, 257, grad_dtype=BF16, momentum=0.0)
    op(g, out=g)
    _check(g, want, BF16)


def test_captured_and_replayed():
    rng = np.random.default_rng(13)
    g, b = _grad(rng, 400, 260), _grad(rng, 400, 260)
    op = tw.Orthogonalize(400, 260)
    eager = tw.Orthogonalize(400, 260)
    b2 = b.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        op(g, b.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = op(g, b)
    for i in range(3):
        g.copy_(_grad(np.random.default_rng(20 + i), 400, 260))
        graph.replay()
        want = eager(g, b2)
        assert torch.equal(out, want) and torch.equal(b, b2)


def test_on_a_side_stream():
    g = _grad(np.random.default_rng(14), 256, 300)
    op = tw.Orthogonalize(256, 300, momentum=0.0)
    want = op(g).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.zeros(1 << 26, device="cuda").add_(1)  # keeps the stream busy
        later = g * 1.0
        got = op(later)
    s.synchronize()
    assert torch.equal(got, want) and big[0] == 1


def test_one_shot():
    g = _grad(np.random.default_rng(15), 70, 50)
    out, status = tw.orthogonalize(g, scale=2.0)
    assert status.item() == 0
    _check(out, 2.0 * updates.newton_schulz(_f64(g)), BF16)


def _exact(g, steps=5, coefficients=updates.COEFFICIENTS):
    """updates.newton_schulz on the GPU, for sizes that numpy would take long over."""
    x = g.double()
    x = x / x.norm()
    a, b, c = coefficients
    for _ in range(steps):
        gram = x.T @ x if x.shape[0] >= x.shape[1] else x @ x.T
        p = b * gram + c * gram @ gram
        x = a * x + (x @ p if x.shape[0] >= x.shape[1] else p @ x)
    return x.cpu().numpy()


# tall and thin (many slices of a tile), more tiles than pairs of SMs, the layer's own shapes
@pytest.mark.parametrize("m,n,count", [(70000, 40, 1), (40, 70000, 2), (9000, 300, 1), (3000, 2900, 1), (5632, 2048, 1), (2048, 8192, 2)])
def test_large(m, n, count):
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    gs = [torch.randn(m, n, generator=gen, device="cuda") * torch.exp(torch.randn(m, 1, generator=gen, device="cuda")) for _ in range(count)]
    op = tw.Orthogonalize(m, n, count=count, momentum=0.0)
    outs = op(gs)
    torch.cuda.synchronize()
    tw.raise_if_device_error(op.status)
    for g, o in zip(gs, outs):
        _check(o, _exact(g), BF16)


def test_two_at_once_on_two_streams():
    """Neither waits for the other's units, and neither is disturbed."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    sizes = [(2000, 1500), (1300, 2100)]
    gs = [torch.randn(*s, generator=gen, device="cuda") for s in sizes]
    ops = [tw.Orthogonalize(*s, momentum=0.0) for s in sizes]
    want = [op(g).clone() for op, g in zip(ops, gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(ops[i](gs[i]).clone())
    torch.cuda.synchronize()
    for i in range(2):
        tw.raise_if_device_error(ops[i].status)
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_next_to_other_work_on_the_gpu():
    """Long kernels on another stream hold SMs back from the products."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    g = torch.randn(2048, 1024, generator=gen, device="cuda")
    op = tw.Orthogonalize(2048, 1024, momentum=0.0)
    want = op(g).clone()
    a = torch.randn(8192, 8192, device="cuda", dtype=BF16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(30):
            b = a @ a
    for _ in range(10):
        assert torch.equal(op(g), want)
    torch.cuda.synchronize()
    tw.raise_if_device_error(op.status)
    assert b.shape == a.shape
