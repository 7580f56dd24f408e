"""GPU parity of layer norm, forward and backward, against oracle/ends.py in float64.

Tolerances, from the arithmetic (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32, one rounding of
each result; fp32 inside):
* a row sum is at most 16 sequential terms a thread and two five-level trees, so its
  error is at most 26 * 2^-24 of the sum of magnitudes; the mean's, the variance's and
  the products' roundings together stay below F = 64 * 2^-24 of a result's terms:
  |y - ref| <= u |ref| + F ((|s| + mean|s|) rstd |w| + |b|), and for dx the same with
  its own terms;
* dweight and dbias sum T products in fp32, sequentially within a CTA at worst:
  F + T 2^-24 of the sum of magnitudes, whose typical size is far smaller.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import ends  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
F = 64 * 2.0 ** -24
EPS = 1e-5
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _rand(rng, shape, dtype, loc=0.0, scale=1.0):
    return torch.from_numpy(rng.normal(loc, scale, shape).astype(np.float32)).to(dtype).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, tol, what):
    got = _f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} against {ref[bad][0]}"


def _check_fwd(y, s, w, b, mean, rstd, dtype):
    S = _f64(s)
    W = np.ones(S.shape[1]) if w is None else _f64(w)
    B = np.zeros(S.shape[1]) if b is None else _f64(b)
    ry, rm, rr = ends.layer_norm(S, W, B, EPS)
    mag = np.abs(S).mean(axis=1)
    _close(mean, rm, F * mag + 1e-30, "mean")
    # the variance's error is F of it plus the mean's squared error, over 2 in the root
    _close(rstd, rr, rr * (F + (F * mag * rr) ** 2), "rstd")
    terms = (np.abs(S) + mag[:, None]) * rr[:, None] * np.abs(W) + np.abs(B)
    _close(y, ry, U[dtype] * np.abs(ry) + F * terms + TINY[dtype], "y")


SHAPES = [(1, 1), (1, 7), (2, 31), (3, 256), (5, 1027), (77, 2048), (130, 2047), (17, 4096), (9, 8192), (6, 8200),
          (3, 16384), (700, 512), (2000, 96), (330, 1000), (400, 2040), (350, 4096), (330, 5632), (330, 8192), (330, 9000),
          (100, 1027), (90, 8199), (321, 16384), (2500, 500), (1100, 1288), (700, 2400), (330, 2600), (330, 5120), (340, 6400),
          (330, 7168)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,residual", [(BF16, F32, True), (BF16, BF16, False), (F16, F16, True), (F32, F32, False),
                                                   (F16, F32, False), (F32, F32, True)])
def test_forward_matches_oracle(T, d, dtype, wdtype, residual):
    rng = np.random.default_rng(T * 31 + d)
    x, w, b = _rand(rng, (T, d), dtype, 0.3, 1.5), _rand(rng, d, wdtype, 1, 0.3), _rand(rng, d, wdtype, 0, 0.2)
    r = _rand(rng, (T, d), dtype, -0.2, 2.0) if residual else None
    ln = tw.LayerNorm(T, d, dtype=dtype, weight_dtype=wdtype, eps=EPS)
    y, s = ln.forward(x, w, b, residual=r)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
    else:
        assert s is x
    _check_fwd(y, s, w, b, ln.mean, ln.rstd, dtype)


def _check_bwd(dx, dw, db, dy, x, w, dres, mean, rstd, dtype):
    X, DY, M, R = _f64(x), _f64(dy), _f64(mean)[:, None], _f64(rstd)[:, None]
    T, d = X.shape
    W = np.ones(d) if w is None else _f64(w)
    xh = (X - M) * R
    g = DY * W
    ref = R * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    axh = (np.abs(X) + np.abs(M)) * R
    terms = R * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + axh * (np.abs(g) * axh).mean(1, keepdims=True))
    if dres is not None:
        ref = ref + _f64(dres)
        terms = terms + np.abs(_f64(dres))
    _close(dx, ref, U[dtype] * np.abs(ref) + F * terms + TINY[dtype], "dx")
    over_rows = F + T * 2.0 ** -24
    _close(dw, (DY * xh).sum(0), over_rows * (np.abs(DY) * axh).sum(0), "dweight")
    _close(db, DY.sum(0), over_rows * np.abs(DY).sum(0), "dbias")
    # and the definition end to end, in norm: the statistics' fp32 errors are far below this
    full, fw, fb = ends.layer_norm_grad(DY, X, W, EPS, None if dres is None else _f64(dres))
    for got, want, u in ((dx, full, U[dtype]), (dw, fw, 2.0 ** -24), (db, fb, 2.0 ** -24)):
        if d > 1:  # a single column's dx and dweight are 0: nothing to be relative to
            assert np.linalg.norm(_f64(got) - want) <= (u + 1e-5) * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,residual", [(BF16, F32, True), (BF16, BF16, False), (F16, F16, True), (F32, F32, False),
                                                   (F32, F32, True)])
def test_backward_matches_oracle(T, d, dtype, wdtype, residual):
    rng = np.random.default_rng(T * 37 + d)
    x, w = _rand(rng, (T, d), dtype, 0.3, 1.5), _rand(rng, d, wdtype, 1, 0.3)
    dy = _rand(rng, (T, d), dtype, 0, 0.5)
    dres = _rand(rng, (T, d), dtype, 0, 0.5) if residual else None
    ln = tw.LayerNorm(T, d, dtype=dtype, weight_dtype=wdtype, eps=EPS)
    ln.forward(x, w)
    dx, dw, db = ln.backward(dy, x, w, dres=dres)
    torch.cuda.synchronize()
    _check_bwd(dx, dw, db, dy, x, w, dres, ln.mean, ln.rstd, dtype)


def test_without_weight_and_bias():
    rng = np.random.default_rng(2)
    x, dy = _rand(rng, (33, 640), BF16), _rand(rng, (33, 640), BF16)
    y, s, mean, rstd = tw.layer_norm_fwd(x)
    _check_fwd(y, s, None, None, mean, rstd, BF16)
    dx, dw, db = tw.layer_norm_bwd(dy, x, mean, rstd)
    _check_bwd(dx, dw, db, dy, x, None, None, mean, rstd, BF16)


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 0), (3, 1), (5, 2)])
def test_strided_and_unaligned_rows(pad, off):
    rng = np.random.default_rng(pad * 10 + off)
    T, d = 19, 512
    full = _rand(rng, (T, d + pad), BF16)
    x = full[:, min(off, pad):][:, :d]
    dyf = _rand(rng, (T, d + 2 * pad), BF16)
    dy = dyf[:, pad:pad + d]
    w = _rand(rng, d, BF16, 1, 0.3)
    ln = tw.LayerNorm(T, d, weight_dtype=BF16)
    y, _ = ln.forward(x, w)
    _check_fwd(y, x, w, None, ln.mean, ln.rstd, BF16)
    dx, dw, db = ln.backward(dy, x, w)
    _check_bwd(dx, dw, db, dy, x, w, None, ln.mean, ln.rstd, BF16)
    # bits do not depend on where the rows lie when the access width is the same
    if pad == 8:
        ln2 = tw.LayerNorm(T, d, weight_dtype=BF16)
        assert torch.equal(ln2.forward(x.contiguous(), w)[0], y)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d", [(3, 1), (90, 3), (700, 7), (90, 8), (90, 9), (700, 15), (90, 33), (700, 250), (90, 257), (90, 1027), (700, 2050),
                                 (330, 4101), (5, 8190), (330, 9001)])
def test_rows_at_any_offset_touch_their_own_columns_only(dtype, T, d):
    """Inputs between NaN, outputs between nines, each at an offset and a stride of its own."""
    from activation_sparse_feedforward_gb300 import _lib
    rng = np.random.default_rng(T + d)
    w, b = _rand(rng, d, F32, 1, 0.3), _rand(rng, d, F32, 0, 0.2)
    ln = tw.LayerNorm(T, d, dtype=dtype, weight_dtype=F32, eps=EPS)
    dt = {F32: 0, BF16: 1, F16: 2}[dtype]

    def inside(off, pad, fill, values):
        buf = torch.full((T, off + d + pad), fill, dtype=dtype, device="cuda")
        if values is not None:
            buf[:, off:off + d] = values
        return buf, buf[:, off:off + d]

    vals = [_rand(rng, (T, d), dtype, 0.3, 1.5) for _ in range(2)]
    stream = torch.cuda.current_stream().cuda_stream
    for offs in ((0, 1, 2, 3), (1, 6, 0, 5), (7, 3, 4, 1), (2, 2, 2, 2), (3, 0, 6, 4)):
        (_, x), (_, r) = inside(offs[0], offs[1] % 3, float("nan"), vals[0]), inside(offs[1], offs[2] % 5, float("nan"), vals[1])
        (sb, s), (yb, y) = inside(offs[2], offs[3] % 4, 9.0, None), inside(offs[3], offs[0] % 6, 9.0, None)
        code = tw.load().tw_layer_norm_fwd(x.data_ptr(), x.stride(0), r.data_ptr(), r.stride(0), w.data_ptr(), b.data_ptr(), T, d, EPS,
                                           dt, 0, s.data_ptr(), s.stride(0), y.data_ptr(), y.stride(0), ln.mean.data_ptr(),
                                           ln.rstd.data_ptr(), stream)
        assert code == _lib.TW_OK
        assert torch.equal(s, (vals[0].float() + vals[1].float()).to(dtype))
        _check_fwd(y, s, w, b, ln.mean, ln.rstd, dtype)
        (db_, dx), (_, dres) = inside(offs[1], offs[0] % 4, 9.0, None), inside(offs[3], offs[1] % 7, float("nan"), vals[0])
        code = tw.load().tw_layer_norm_bwd(r.data_ptr(), r.stride(0), s.data_ptr(), s.stride(0), ln.mean.data_ptr(), ln.rstd.data_ptr(),
                                           w.data_ptr(), dres.data_ptr(), dres.stride(0), T, d, dt, 0, dx.data_ptr(), dx.stride(0),
                                           ln.dweight.data_ptr(), ln.dbias.data_ptr(), ln.ws.data_ptr(), ln.ws.numel(), stream)
        assert code == _lib.TW_OK
        _check_bwd(dx, ln.dweight, ln.dbias, r, s, w, dres, ln.mean, ln.rstd, dtype)
        for buf, off in ((sb, offs[2]), (yb, offs[3]), (db_, offs[1])):
            assert (buf[:, :off] == 9).all() and (buf[:, off + d:] == 9).all()


@pytest.mark.parametrize("T,d", [(40, 3), (40, 777), (400, 777)])
def test_one_odd_row_for_all(T, d):
    rng = np.random.default_rng(d)
    x, r = _rand(rng, (1, d), BF16).expand(T, d), _rand(rng, (T, d), BF16)
    ln = tw.LayerNorm(T, d)
    y, s = ln.forward(x, residual=r)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    _check_fwd(y, s, None, None, ln.mean, ln.rstd, BF16)
    dx, dw, db = ln.backward(x, s, dres=x)
    _check_bwd(dx, dw, db, x, s, None, x, ln.mean, ln.rstd, BF16)


def test_one_row_for_all_and_fewer_rows_than_the_object():
    rng = np.random.default_rng(5)
    x, r = _rand(rng, (1, 768), BF16).expand(40, 768), _rand(rng, (40, 768), BF16)
    ln = tw.LayerNorm(64, 768)
    y, s = ln.forward(x, residual=r)
    assert y.shape == (40, 768) and ln.mean.shape == (40,)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    _check_fwd(y, s, None, None, ln.mean, ln.rstd, BF16)
    dx, dw, db = ln.backward(r, s)
    assert dx.shape == (40, 768)
    _check_bwd(dx, dw, db, r, s, None, None, ln.mean, ln.rstd, BF16)


def test_in_place_stream_and_gradient():
    """The residual stream may be updated in place (sum = res) and dx may replace dres."""
    from activation_sparse_feedforward_gb300 import _lib
    rng = np.random.default_rng(6)
    T, d = 50, 2048
    x, r, w = _rand(rng, (T, d), BF16), _rand(rng, (T, d), BF16), _rand(rng, d, F32, 1, 0.2)
    ln = tw.LayerNorm(T, d, weight_dtype=F32)
    y, s = (t.clone() for t in ln.forward(x, w, residual=r))
    y2, stream = torch.empty_like(y), r.clone()
    st = torch.cuda.current_stream().cuda_stream
    L = tw.load()
    code = L.tw_layer_norm_fwd(x.data_ptr(), d, stream.data_ptr(), d, w.data_ptr(), None, T, d, 1e-5, 1, 0,
                               stream.data_ptr(), d, y2.data_ptr(), d, None, None, st)
    assert code == _lib.TW_OK
    assert torch.equal(stream, s) and torch.equal(y2, y)
    dy, dres = _rand(rng, (T, d), BF16), _rand(rng, (T, d), BF16)
    dx, dw, _ = (t.clone() for t in ln.backward(dy, s, w, dres=dres))
    g = dres.clone()
    dw2 = torch.empty_like(dw)
    code = L.tw_layer_norm_bwd(dy.data_ptr(), d, s.data_ptr(), d, ln.mean.data_ptr(), ln.rstd.data_ptr(), w.data_ptr(),
                               g.data_ptr(), d, T, d, 1, 0, g.data_ptr(), d, dw2.data_ptr(), None, ln.ws.data_ptr(),
                               ln.ws.numel(), st)
    assert code == _lib.TW_OK
    assert torch.equal(g, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("T", [5, 77, 400, 1500])
@pytest.mark.parametrize("d", [777, 2048])
def test_gradient_in_place_of_its_input(T, d):
    """dx over dy, and over x: the sums over rows still see the inputs."""
    from activation_sparse_feedforward_gb300 import _lib
    rng = np.random.default_rng(T + d)
    x, dy, w = _rand(rng, (T, d), BF16), _rand(rng, (T, d), BF16), _rand(rng, d, F32, 1, 0.2)
    ln = tw.LayerNorm(T, d, weight_dtype=F32)
    ln.forward(x, w)
    for over in ("dy", "x"):
        t = dict(x=x.clone(), dy=dy.clone())
        code = tw.load().tw_layer_norm_bwd(t["dy"].data_ptr(), d, t["x"].data_ptr(), d, ln.mean.data_ptr(),
                                           ln.rstd.data_ptr(), w.data_ptr(), None, 0, T, d, 1, 0, t[over].data_ptr(), d,
                                           ln.dweight.data_ptr(), ln.dbias.data_ptr(), ln.ws.data_ptr(), ln.ws.numel(),
                                           torch.cuda.current_stream().cuda_stream)
        assert code == _lib.TW_OK
        _check_bwd(t[over], ln.dweight, ln.dbias, dy, x, w, None, ln.mean, ln.rstd, BF16)


def test_rows_are_independent_and_nan_stays_in_its_row():
    rng = np.random.default_rng(7)
    x = _rand(rng, (12, 1024), BF16)
    clean = tw.layer_norm_fwd(x)[0]
    bad = x.clone()
    bad[3, 17] = float("nan")
    bad[8, 0] = float("inf")
    y = tw.layer_norm_fwd(bad)[0]
    assert torch.isnan(y[3]).all() and torch.isnan(y[8]).all()
    keep = [i for i in range(12) if i not in (3, 8)]
    assert torch.equal(y[keep], clean[keep])


def test_constant_rows_and_large_offsets():
    """Variance 0 gives the bias; a mean of 1000 standard deviations keeps the two-sweep
    variance's precision (a sum of squares in fp32 would lose it all)."""
    d = 1536
    b = torch.linspace(-1, 1, d, device="cuda")
    y = tw.layer_norm_fwd(torch.full((5, d), 3.0, device="cuda"), None, b)[0]
    assert torch.equal(y, b.expand(5, d))
    rng = np.random.default_rng(8)
    x = _rand(rng, (7, d), F32, 1000.0, 1.0)
    y, s, mean, rstd = tw.layer_norm_fwd(x)
    ref = ends.layer_norm(_f64(x), eps=EPS)
    _close(rstd, ref[2], 1e-4 * ref[2], "rstd")
    _check_fwd(y, s, None, None, mean, rstd, F32)


def test_no_rows():
    ln = tw.LayerNorm(4, 256)
    e = torch.empty(0, 256, dtype=BF16, device="cuda")
    ln.dweight.fill_(7)
    ln.dbias.fill_(7)
    assert ln.forward(e)[0].shape == (0, 256)
    dx, dw, db = ln.backward(e, e)
    assert dx.shape == (0, 256) and not dw.any() and not db.any()


def test_gradient_against_differences_of_the_forward():
    """Along random directions, with the fp32 kernel itself: (L(x + h v) - L(x - h v)) / 2h.
    The forward's fp32 error over h leaves about 2^-22 sqrt(d) / h, the truncation h^2."""
    rng = np.random.default_rng(9)
    T, d, h = 6, 900, 1e-2
    x, w, dy = _rand(rng, (T, d), F32), _rand(rng, d, F32, 1, 0.3), _rand(rng, (T, d), F32)
    _, _, mean, rstd = tw.layer_norm_fwd(x, w)
    dx, dw, _ = tw.layer_norm_bwd(dy, x, mean, rstd, w)

    def loss(xv, wv):
        return (tw.layer_norm_fwd(xv, wv)[0].double() * dy.double()).sum().item()

    for k in range(3):
        v, u = _rand(rng, (T, d), F32), _rand(rng, d, F32)
        num = (loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h)
        ref = (dx.double() * v.double()).sum().item()
        assert abs(num - ref) <= 2e-3 * (abs(ref) + dx.double().norm().item())
        num = (loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h)
        ref = (dw.double() * u.double()).sum().item()
        assert abs(num - ref) <= 2e-3 * (abs(ref) + dw.double().norm().item())


@pytest.mark.parametrize("T,d", [(3, 640), (5000, 2048), (300, 1027)])
def test_same_bits_every_time_and_on_another_stream(T, d):
    rng = np.random.default_rng(10)
    x, dy = _rand(rng, (T, d), BF16), _rand(rng, (T, d), BF16)
    ln = tw.LayerNorm(T, d)
    y = ln.forward(x)[0].clone()
    first = [t.clone() for t in ln.backward(dy, x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = ln.forward(x)[0].clone()
        again = [t.clone() for t in ln.backward(dy, x)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_in_a_graph():
    rng = np.random.default_rng(11)
    x, r, dy = (_rand(rng, (100, 2048), BF16) for _ in range(3))
    ln = tw.LayerNorm(100, 2048)
    y, s = ln.forward(x, residual=r)
    want = [t.clone() for t in (y, s, *ln.backward(dy, s))]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, s = ln.forward(x, residual=r)
        got = (y, s, *ln.backward(dy, s))
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
