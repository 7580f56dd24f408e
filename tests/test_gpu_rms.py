"""GPU parity of root-mean-square norm, forward (into the type and into 8 bits) and backward,
against oracle/ends.py in float64.

Tolerances, from the arithmetic (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32, one rounding of each
result; fp32 inside): a row's sum is at most 16 sequential terms a thread and two five-level
trees, with the products' roundings and the root's below F = 64 * 2^-24 of a result's terms.
dweight sums T products in fp32, sequentially within a CTA at worst: F + T 2^-24 of the sum
of magnitudes.
8 bits: the scale is F off at most; q is the e4m3 number nearest to y / scale, whose own error
is 2 F, so that next to a border the other neighbour is right too: q must equal the rounding
of a value within 2 F of the oracle's.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402
from oracle import ends  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
F = 64 * 2.0 ** -24
EPS = 1e-6
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CODE = {F32: 0, BF16: 1, F16: 2}


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


def _ref(s, w):
    W = np.ones(s.shape[1]) if w is None else _f64(w)
    return ends.rms_norm(_f64(s), W, EPS)


def _check_fwd(y, s, w, rstd, dtype):
    ry, rr = _ref(s, w)
    _close(rstd, rr, rr * F, "rstd")
    _close(y, ry, U[dtype] * np.abs(ry) + F * np.abs(ry) + TINY[dtype], "y")


def _check_fp8(q, scales, s, w, rstd, group):
    ry, rr = _ref(s, w)
    _close(rstd, rr, rr * F, "rstd")
    rs = ends.fp8_scales(ry, group)
    _close(scales, rs, rs * F, "scales")
    wide = rs if group == 0 else np.repeat(rs, group, axis=1)[:, :ry.shape[1]]
    v = ry / wide
    got = _f64(q)
    ok = (got >= ends.to_e4m3(v - 2 * F * np.abs(v))) & (got <= ends.to_e4m3(v + 2 * F * np.abs(v)))
    assert ok.all(), f"{(~ok).sum()} of {ok.size} q outside; first at {np.argwhere(~ok)[0]}: {got[~ok][0]} for {v[~ok][0]}"


SHAPES = [(1, 1), (1, 7), (2, 31), (3, 256), (5, 1027), (77, 2048), (130, 2047), (17, 4096), (9, 8192), (6, 8200),
          (3, 16384), (700, 512), (2000, 96), (330, 1000), (400, 2040), (350, 4096), (330, 5632), (330, 8192), (330, 9000),
          (100, 1027), (90, 8199), (321, 16384), (2500, 500), (1100, 1288), (700, 2400), (330, 2600), (330, 5120), (340, 6400),
          (330, 7168), (1, 64), (13, 128), (4001, 64), (1203, 128), (3331, 120), (2505, 200), (1027, 256), (90001, 8)]
TYPES = [(BF16, F32, True), (BF16, BF16, False), (F16, F16, True), (F32, F32, False), (F16, F32, False), (F32, F32, True)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,residual", TYPES)
@pytest.mark.parametrize("out", ["same", "row", "group"])
def test_forward_matches_oracle(T, d, dtype, wdtype, residual, out):
    rng = np.random.default_rng(T * 31 + d)
    x, w = _rand(rng, (T, d), dtype, 0.3, 1.5), _rand(rng, d, wdtype, 1, 0.3)
    r = _rand(rng, (T, d), dtype, -0.2, 2.0) if residual else None
    group = 128 if out == "group" else 0
    op = tw.RMSNorm(T, d, dtype=dtype, weight_dtype=wdtype, eps=EPS, fp8=out != "same", group=group, backward=False)
    res = op.forward(x, w, residual=r) if out == "same" else op.forward_fp8(x, w, residual=r)
    torch.cuda.synchronize()
    s = res[-1]
    if residual:
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
    else:
        assert s is x
    if out == "same":
        _check_fwd(res[0], s, w, op.rstd, dtype)
    else:
        _check_fp8(res[0], res[1], s, w, op.rstd, group)


def _check_bwd(dx, dw, dy, x, w, dres, rstd, dtype):
    X, DY, R = _f64(x), _f64(dy), _f64(rstd)[:, None]
    T, d = X.shape
    W = np.ones(d) if w is None else _f64(w)
    xh, g = X * R, DY * W
    ref = R * (g - xh * (g * xh).mean(1, keepdims=True))
    terms = R * (np.abs(g) + np.abs(xh) * (np.abs(g) * np.abs(xh)).mean(1, keepdims=True))
    if dres is not None:
        ref, terms = ref + _f64(dres), terms + np.abs(_f64(dres))
    _close(dx, ref, U[dtype] * np.abs(ref) + F * terms + TINY[dtype], "dx")
    _close(dw, (DY * xh).sum(0), (F + T * 2.0 ** -24) * (np.abs(DY) * np.abs(xh)).sum(0), "dweight")
    # and the definition end to end, in norm
    full, fw = ends.rms_norm_grad(DY, X, W, EPS, None if dres is None else _f64(dres))
    for got, want, u in ((dx, full, U[dtype]), (dw, fw, 2.0 ** -24)):
        if d > 1:  # a single column's dx is 0 but for eps: nothing to be relative to
            assert np.linalg.norm(_f64(got) - want) <= (u + 1e-5) * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,residual", [t for t in TYPES if t != (F16, F32, False)])
def test_backward_matches_oracle(T, d, dtype, wdtype, residual):
    rng = np.random.default_rng(T * 37 + d)
    x, w = _rand(rng, (T, d), dtype, 0.3, 1.5), _rand(rng, d, wdtype, 1, 0.3)
    dy = _rand(rng, (T, d), dtype, 0, 0.5)
    dres = _rand(rng, (T, d), dtype, 0, 0.5) if residual else None
    op = tw.RMSNorm(T, d, dtype=dtype, weight_dtype=wdtype, eps=EPS)
    op.forward(x, w)
    dx, dw = op.backward(dy, x, w, dres=dres)
    torch.cuda.synchronize()
    _check_bwd(dx, dw, dy, x, w, dres, op.rstd, dtype)
    again = tw.RMSNorm(T, d, dtype=dtype, weight_dtype=wdtype, eps=EPS).backward(dy, x, w, dres=dres, rstd=op.rstd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_without_weight():
    rng = np.random.default_rng(2)
    x, dy = _rand(rng, (33, 640), BF16), _rand(rng, (33, 640), BF16)
    y, s, rstd = tw.rms_norm_fwd(x)
    _check_fwd(y, s, None, rstd, BF16)
    q, scales, s, rstd = tw.rms_norm_fwd_fp8(x, group=128)
    _check_fp8(q, scales, s, None, rstd, 128)
    dx, dw = tw.rms_norm_bwd(dy, x, rstd)
    _check_bwd(dx, dw, dy, x, None, None, rstd, BF16)


def test_fewer_rows_than_the_object_was_made_for():
    rng = np.random.default_rng(3)
    x, w = _rand(rng, (7, 256), BF16), _rand(rng, 256, BF16)
    op = tw.RMSNorm(20, 256)
    op.y.fill_(9)
    y, _ = op.forward(x, w)
    assert y.shape == (7, 256) and op.rstd.shape == (7,) and (op.y[7:] == 9).all()
    _check_fwd(y, x, w, op.rstd, BF16)
    dx, dw = op.backward(x, x, w)
    _check_bwd(dx, dw, x, x, w, None, op.rstd, BF16)
    dx, dw = tw.RMSNorm(20, 256).backward(x[:0], x[:0], w, rstd=op.rstd[:0])
    assert dx.shape == (0, 256) and not dw.any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d", [(3, 1), (90, 3), (700, 7), (90, 8), (700, 15), (90, 33), (700, 250), (90, 257), (90, 1027), (700, 2050),
                                 (330, 4101), (5, 8190), (330, 9001)])
def test_rows_at_any_offset_touch_their_own_columns_only(dtype, T, d):
    """Inputs between NaN, outputs between nines, each at an offset and a stride of its own."""
    rng = np.random.default_rng(T + d)
    w = _rand(rng, d, F32, 1, 0.3)
    op = tw.RMSNorm(T, d, dtype=dtype, weight_dtype=F32, eps=EPS)
    scales = torch.empty((T, (d + 127) // 128), device="cuda")
    lib, dt = tw.load(), CODE[dtype]

    def inside(off, pad, fill, values, dt_=None):
        buf = torch.full((T, off + d + pad), fill, dtype=dt_ or dtype, device="cuda")
        if values is not None:
            buf[:, off:off + d] = values
        return buf, buf[:, off:off + d]

    vals = [_rand(rng, (T, d), dtype, 0.3, 1.5) for _ in range(2)]
    stream = torch.cuda.current_stream().cuda_stream
    for offs in ((0, 1, 2, 3), (1, 6, 0, 5), (7, 3, 4, 1), (2, 2, 2, 2), (8, 0, 6, 8)):
        (_, x), (_, r) = inside(offs[0], offs[1] % 3, float("nan"), vals[0]), inside(offs[1], offs[2] % 5, float("nan"), vals[1])
        (sb, s), (yb, y) = inside(offs[2], offs[3] % 4, 9.0, None), inside(offs[3], offs[0] % 6, 9.0, None)
        common = x.data_ptr(), x.stride(0), r.data_ptr(), r.stride(0), w.data_ptr(), T, d, EPS, dt, 0, s.data_ptr(), s.stride(0)
        assert lib.tw_rms_norm_fwd(*common, y.data_ptr(), y.stride(0), op.rstd.data_ptr(), stream) == _lib.TW_OK
        assert torch.equal(s, (vals[0].float() + vals[1].float()).to(dtype))
        _check_fwd(y, s, w, op.rstd, dtype)
        for group in (0, 128):
            qb, q = inside(offs[3], offs[1] % 6, 9, None, torch.uint8)
            sc = scales if group else scales.view(-1)[:T].view(T, 1)
            assert lib.tw_rms_norm_fwd_fp8(*common, q.data_ptr(), q.stride(0), sc.data_ptr(), group, op.rstd.data_ptr(),
                                           stream) == _lib.TW_OK
            _check_fp8(q.contiguous().view(torch.float8_e4m3fn), sc, s, w, op.rstd, group)
            assert (qb[:, :offs[3]] == 9).all() and (qb[:, offs[3] + d:] == 9).all()
        (db, dx), (_, dres) = inside(offs[1], offs[0] % 4, 9.0, None), inside(offs[3], offs[1] % 7, float("nan"), vals[0])
        code = lib.tw_rms_norm_bwd(r.data_ptr(), r.stride(0), s.data_ptr(), s.stride(0), op.rstd.data_ptr(), w.data_ptr(),
                                   dres.data_ptr(), dres.stride(0), T, d, dt, 0, dx.data_ptr(), dx.stride(0),
                                   op.dweight.data_ptr(), op.ws.data_ptr(), op.ws_bytes, stream)
        assert code == _lib.TW_OK
        _check_bwd(dx, op.dweight, r, s, w, dres, op.rstd, dtype)
        for buf, off in ((sb, offs[2]), (yb, offs[3]), (db, offs[1])):
            assert (buf[:, :off] == 9).all() and (buf[:, off + d:] == 9).all()


@pytest.mark.parametrize("T,d", [(40, 3), (40, 777), (400, 777), (400, 1024)])
def test_one_row_for_all(T, d):
    rng = np.random.default_rng(d)
    x, r = _rand(rng, (1, d), BF16).expand(T, d), _rand(rng, (T, d), BF16)
    op = tw.RMSNorm(T, d)
    y, s = op.forward(x, residual=r)
    assert torch.equal(s, (x.float() + r.float()).bfloat16())
    _check_fwd(y, s, None, op.rstd, BF16)


@pytest.mark.parametrize("d", [512, 777])
@pytest.mark.parametrize("group", [0, 128])
def test_nan_infinity_and_zero_rows(d, group):
    x = _rand(np.random.default_rng(5), (6, d), BF16)
    x[1, 3], x[2, 300], x[3], x[4, 0] = float("nan"), float("inf"), 0.0, -float("inf")
    op = tw.RMSNorm(6, d, fp8=True, group=group, backward=False)
    q, scales, _ = op.forward_fp8(x)
    y, _, _ = tw.rms_norm_fwd(x)
    for t in (0, 5):
        _check_fp8(q[t:t + 1], scales[t:t + 1], x[t:t + 1], None, op.rstd[t:t + 1], group)
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all() and torch.isnan(scales[1]).all()
    assert not q[3].float().any() and (scales[3] == 2.0 ** -126).all()
    for t, c in ((2, 300), (4, 0)):  # 0 times infinity in that column, finite values times 0 elsewhere
        assert torch.isnan(y[t, c]) and torch.isnan(q[t, c].float()) and torch.isnan(scales[t, c // 128 if group else 0])
        if group:
            keep = torch.ones(d, dtype=torch.bool)
            keep[c // 128 * 128:c // 128 * 128 + 128] = False
            assert not q[t].float().cpu()[keep].any()


def test_a_nan_weight_reaches_its_scale():
    x, w = _rand(np.random.default_rng(6), (3, 512), BF16), torch.ones(512, dtype=BF16, device="cuda")
    w[200] = float("nan")
    q, scales, _, _ = tw.rms_norm_fwd_fp8(x, w)
    assert torch.isnan(scales).all()
    q, scales, _, _ = tw.rms_norm_fwd_fp8(x, w, group=128)
    assert torch.isnan(scales[:, 1]).all() and torch.isfinite(scales[:, [0, 2, 3]]).all()


def test_large_and_small_magnitudes_in_8_bits():
    rng = np.random.default_rng(7)
    x, w = _rand(rng, (20, 1024), F32), _rand(rng, 1024, F32, 0, 1e-30)
    q, scales, s, rstd = tw.rms_norm_fwd_fp8(x, w, group=128)
    _check_fp8(q, scales, s, w, rstd, 128)
    q, scales, s, rstd = tw.rms_norm_fwd_fp8(x, w * 1e60)  # infinite in fp32: no scale holds it
    assert torch.isinf(scales).all() and torch.isnan(q.float()).all()
    w = _rand(rng, 1024, F32, 0, 1e30)
    q, scales, s, rstd = tw.rms_norm_fwd_fp8(x, w)
    _check_fp8(q, scales, s, w, rstd, 0)


def test_in_place():
    rng = np.random.default_rng(8)
    T, d = 400, 1027
    x, r, w = _rand(rng, (T, d), BF16), _rand(rng, (T, d), BF16), _rand(rng, d, BF16)
    lib, stream = tw.load(), torch.cuda.current_stream().cuda_stream
    want = (x.float() + r.float()).bfloat16()
    rstd, y = torch.empty(T, device="cuda"), torch.empty_like(x)
    xx = x.clone()
    assert lib.tw_rms_norm_fwd(xx.data_ptr(), d, r.data_ptr(), d, w.data_ptr(), T, d, EPS, 1, 1, xx.data_ptr(), d, y.data_ptr(),
                               d, rstd.data_ptr(), stream) == _lib.TW_OK
    assert torch.equal(xx, want)
    _check_fwd(y, want, w, rstd, BF16)
    op = tw.RMSNorm(T, d)
    for which in ("dy", "x", "dres"):
        dy, xi, dres = r.clone(), want.clone(), x.clone()
        to = {"dy": dy, "x": xi, "dres": dres}[which]
        assert lib.tw_rms_norm_bwd(dy.data_ptr(), d, xi.data_ptr(), d, rstd.data_ptr(), w.data_ptr(), dres.data_ptr(), d, T, d, 1, 1,
                                   to.data_ptr(), d, op.dweight.data_ptr(), op.ws.data_ptr(), op.ws_bytes, stream) == _lib.TW_OK
        _check_bwd(to, op.dweight, r, want, w, x, rstd, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [8, 64, 72, 128, 256])
def test_short_rows_of_one_warp_know_nothing_of_each_other(dtype, d):
    """Rows of NaN and of zeros next to others, at every number of rows that leaves a warp in part."""
    rng = np.random.default_rng(d)
    full, w = _rand(rng, (345, d), dtype, 0.3, 1.5), _rand(rng, d, dtype, 1, 0.3)
    full[3], full[5] = float("nan"), 0.0
    dy = _rand(rng, (345, d), dtype)
    for T in (*range(321, 346), 1, 2, 6, 17):
        x, op = full[:T], tw.RMSNorm(T, d, dtype=dtype, eps=EPS)
        keep = torch.arange(T, device="cuda") != 3
        y, _ = op.forward(x, w)
        _check_fwd(y[keep], x[keep], w, op.rstd[keep], dtype)
        assert T <= 3 or torch.isnan(y[3]).all()
        op8 = tw.RMSNorm(T, d, dtype=dtype, eps=EPS, fp8=True, group=128, backward=False)
        q, scales, _ = op8.forward_fp8(x, w)
        _check_fp8(q.view(torch.uint8)[keep].view(torch.float8_e4m3fn), scales[keep], x[keep], w, op8.rstd[keep], 128)
        clean = torch.where(torch.isnan(x), torch.full_like(x, 0.25), x)
        op.forward(clean, w)
        dx, dw = op.backward(dy[:T], clean, w)
        _check_bwd(dx, dw, dy[:T], clean, w, None, op.rstd, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,d", [(512, 9), (513, 250), (900, 515), (1300, 1027), (700, 2047), (600, 4101), (520, 6401), (530, 7160),
                                 (520, 8183), (520, 8184), (515, 8185)])
@pytest.mark.parametrize("offset,pad,in_place", [(0, 0, False), (3, 0, True), (5, 2, False), (1, 6, True)])
def test_rows_that_lie_alike(dtype, T, d, offset, pad, in_place):
    """Rows off 16 bytes at one offset and stride in all matrices, whose first and last 16 bytes
    they share with their neighbours: what stands between rows (NaN) and in a row of NaN stays
    out of the others, and nothing else is written."""
    rng = np.random.default_rng(T + d + offset)
    lib, dt, ld = tw.load(), CODE[dtype], d + pad
    stream = torch.cuda.current_stream().cuda_stream
    w = _rand(rng, d, dtype, 1, 0.3)

    def rows(values, fill):
        buf = torch.full((offset + T * ld + 8,), fill, dtype=dtype, device="cuda")
        view = torch.as_strided(buf, (T, d), (ld, 1), offset)
        if values is not None:
            view.copy_(values)
        return buf, view

    def untouched(buf, view):
        view.fill_(9.0)
        return bool((buf == 9).all())

    nan = float("nan")
    vx, vr, vd = (_rand(rng, (T, d), dtype, 0.3, 1.5) for _ in range(3))
    vx[7] = nan
    keep = torch.arange(T, device="cuda") != 7
    (_, x), (_, r), (sb, sm), (yb, y) = rows(vx, nan), rows(vr, nan), rows(None, 9.0), rows(None, 9.0)
    rstd = torch.empty(T, device="cuda")
    fwd = x.data_ptr(), ld, r.data_ptr(), ld, w.data_ptr(), T, d, EPS, dt, dt, sm.data_ptr(), ld
    assert lib.tw_rms_norm_fwd(*fwd, y.data_ptr(), ld, rstd.data_ptr(), stream) == _lib.TW_OK
    want = (vx.float() + vr.float()).to(dtype)
    assert torch.equal(sm[keep], want[keep]) and torch.isnan(y[7]).all()
    _check_fwd(y[keep], want[keep], w, rstd[keep], dtype)
    assert untouched(yb, y)
    qb, scales = torch.full((T, d + 3), 9, dtype=torch.uint8, device="cuda"), torch.empty((T, 1), device="cuda")
    q = qb[:, :d]
    assert lib.tw_rms_norm_fwd_fp8(*fwd, q.data_ptr(), d + 3, scales.data_ptr(), 0, rstd.data_ptr(), stream) == _lib.TW_OK
    _check_fp8(q.contiguous()[keep].view(torch.float8_e4m3fn), scales[keep], want[keep], w, rstd[keep], 0)
    assert (qb[:, d:] == 9).all()

    # backward, of the rows without NaN; dx in the place of dy or of its own
    want[7], rstd[7] = 0.5, 2.0
    sm.copy_(want)
    dres = rows(vr, nan)[1]
    db, dy = rows(vd, 9.0 if in_place else nan)
    if in_place:
        dx = dy
    else:
        db, dx = rows(None, 9.0)
    op = tw.RMSNorm(T, d, dtype=dtype)
    code = lib.tw_rms_norm_bwd(dy.data_ptr(), ld, sm.data_ptr(), ld, rstd.data_ptr(), w.data_ptr(), dres.data_ptr(), ld, T, d, dt, dt,
                               dx.data_ptr(), ld, op.dweight.data_ptr(), op.ws.data_ptr(), op.ws_bytes, stream)
    assert code == _lib.TW_OK
    assert not torch.isnan(dx).any() and not torch.isnan(op.dweight).any()
    k = keep.nonzero()[:, 0]
    X, DY, R, W = _f64(want), _f64(vd), _f64(rstd)[:, None], _f64(w)
    xh = X * R
    _close(op.dweight, (DY * xh).sum(0), (F + T * 2.0 ** -24) * (np.abs(DY) * np.abs(xh)).sum(0), "dweight")
    g = DY * W
    ref = R * (g - xh * (g * xh).mean(1, keepdims=True)) + _f64(vr)
    terms = R * (np.abs(g) + np.abs(xh) * (np.abs(g) * np.abs(xh)).mean(1, keepdims=True)) + np.abs(_f64(vr))
    _close(dx[k], ref[_f64(k).astype(int)], (U[dtype] * np.abs(ref) + F * terms + TINY[dtype])[_f64(k).astype(int)], "dx")
    assert untouched(db, dx) and untouched(sb, sm)


def test_captured_and_replayed():
    rng = np.random.default_rng(9)
    x, w, r = _rand(rng, (64, 512), BF16), _rand(rng, 512, BF16), _rand(rng, (64, 512), BF16)
    op, op8 = tw.RMSNorm(64, 512), tw.RMSNorm(64, 512, fp8=True, backward=False)
    op.forward(x, w, residual=r), op8.forward_fp8(x, w), op.backward(x, r, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = op.forward(x, w, residual=r)
        q, scales, _ = op8.forward_fp8(x, w)
        dx, dw = op.backward(x, s, w)
    x.copy_(_rand(rng, (64, 512), BF16))
    graph.replay()
    _check_fwd(y, s, w, op.rstd, BF16)
    _check_fp8(q, scales, x, w, op8.rstd, 0)
    _check_bwd(dx, dw, x, s, w, None, op.rstd, BF16)
