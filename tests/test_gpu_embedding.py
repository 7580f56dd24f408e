"""GPU parity of the token embedding, forward and backward, against oracle/ends.py in float64.

Tolerances, from the arithmetic (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32): the forward is one
fp32 product (2^-24) and one rounding. The backward adds n rows of a token one after the other,
in parts of at most 1024 rows joined one after the other: n 2^-24 of the sum of magnitudes at
worst, and two roundings for the scale and the addition to what was there.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402
from oracle import ends  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(dtype).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _tokens(rng, T, V, kind):
    if kind == "zipf":
        tok = np.minimum(np.exp(rng.random(T) * np.log(V + 1)).astype(np.int64) - 1, V - 1)
        tok[rng.random(T) < 0.05] = -1
    elif kind == "same":
        tok = np.full(T, V - 1)
    elif kind == "none":
        tok = np.full(T, -1)
    elif kind == "two":
        tok = np.where(rng.random(T) < 0.5, 0, V - 1)
    else:
        tok = rng.integers(0, V, T)
    return tok


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (3, 5, 7), (8, 1000, 2048), (77, 50, 1027), (513, 32000, 64), (40, 300, 8192),
                                   (9, 20, 16384), (2000, 333, 250), (5, 9, 4100)])
@pytest.mark.parametrize("dtype,wdtype,scale", [(BF16, BF16, 1.0), (BF16, F32, 45.25), (F16, F16, 0.3), (F16, F32, 1.0), (F32, F32, 1.7)])
def test_forward_matches_oracle(T, V, d, dtype, wdtype, scale):
    rng = np.random.default_rng(T + V + d)
    tok, w = _tokens(rng, T, V, "zipf"), _rand(rng, (V, d), wdtype, 0.5)
    op = tw.Embedding(T, V, d, dtype=dtype, weight_dtype=wdtype, scale=scale, backward=False)
    y = op.forward(_i32(tok), w)
    torch.cuda.synchronize()
    assert op.status.item() == 0
    ref = ends.embedding(tok, _f64(w), np.float32(scale).astype(np.float64))
    assert (np.abs(_f64(y) - ref) <= (U[dtype] + 2.0 ** -24) * np.abs(ref) + TINY[dtype]).all()
    if dtype == wdtype and scale == 1.0:
        assert torch.equal(y[_i32(tok).long() >= 0], w[_i32(tok[tok >= 0]).long()])


def _check_grad(dw, dy, tok, V, scale, old=None):
    s = float(np.float32(scale))
    ref, mag = ends.embedding_grad(_f64(dy), tok, V, s), ends.embedding_grad(np.abs(_f64(dy)), tok, V, abs(s))
    n = np.bincount(tok[tok >= 0], minlength=V)[:, None]
    tol = (n + 2) * 2.0 ** -24 * mag
    if old is not None:
        ref, tol = ref + _f64(old), tol + 2.0 ** -24 * (np.abs(_f64(old)) + mag)
    bad = ~(np.abs(_f64(dw) - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"
    if old is not None:
        assert torch.equal(dw[_i32(np.nonzero(n[:, 0] == 0)[0]).long()], old[_i32(np.nonzero(n[:, 0] == 0)[0]).long()])


SIZES = [(1, 1, 1), (3, 5, 7), (77, 50, 1027), (512, 700, 96), (513, 700, 96), (700, 100, 2048), (2000, 32, 33), (3000, 5003, 250),
         (1500, 40000, 48), (600, 65, 4100), (530, 20, 16384), (6000, 1024, 16), (5000, 1025, 24)]


@pytest.mark.parametrize("T,V,d", SIZES)
@pytest.mark.parametrize("kind", ["zipf", "same", "two", "uniform", "none"])
@pytest.mark.parametrize("dtype,scale,add", [(BF16, 1.0, False), (F16, 0.5, True), (F32, 45.25, False), (BF16, 2.0, True)])
def test_backward_matches_oracle(T, V, d, kind, dtype, scale, add):
    rng = np.random.default_rng(T * 7 + V + d)
    tok, dy = _tokens(rng, T, V, kind), _rand(rng, (T, d), dtype)
    op = tw.Embedding(T, V, d, dtype=dtype, scale=scale)
    op.dweight.copy_(_rand(rng, (V, d), F32) if add else torch.full((V, d), float("nan"), device="cuda"))
    old = op.dweight.clone() if add else None
    dw = op.backward(dy, _i32(tok), add=add)
    torch.cuda.synchronize()
    assert op.status.item() == 0
    _check_grad(dw, dy, tok, V, scale, old)
    # the same call again gives the same bits, whatever the workspace holds
    if not add:
        first = dw.clone()
        op.ws.fill_(255)
        assert torch.equal(op.backward(dy, _i32(tok)), first)


@pytest.mark.parametrize("T", [150000, 300001])
def test_long_batches(T):
    """Chunks of more than 32 rows; one token of a third of them."""
    rng = np.random.default_rng(T)
    V, d = 900, 16
    tok = np.where(rng.random(T) < 0.3, 17, _tokens(rng, T, V, "zipf"))
    dy = _rand(rng, (T, d), BF16)
    dw, status = tw.embedding_bwd(dy, _i32(tok), V)
    n = np.bincount(tok[tok >= 0], minlength=V)[:, None]
    ref, mag = np.zeros((V, d)), np.zeros((V, d))
    np.add.at(ref, tok[tok >= 0], _f64(dy)[tok >= 0])
    np.add.at(mag, tok[tok >= 0], np.abs(_f64(dy))[tok >= 0])
    assert status.item() == 0 and (np.abs(_f64(dw) - ref) <= (n + 2) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("V", [7, 2000, 60000])
@pytest.mark.parametrize("offset", [0, 1])
def test_batches_whose_stretches_differ(V, offset):
    """One token's positions together, others' anywhere, and a stretch of padding: the parts that
    the sort reads differ in how many of them belong to one range of tokens. Sums of small
    integers are exact in every order."""
    rng = np.random.default_rng(V + offset)
    T, d = 30001, 9
    tok = rng.integers(0, V, T)
    tok[4000:14000], tok[20000:23000] = 5, -1
    dy = rng.integers(-8, 9, (T, d))
    both = torch.from_numpy(np.concatenate([np.zeros(offset, np.int32), tok.astype(np.int32)])).cuda()
    dw, status = tw.embedding_bwd(torch.from_numpy(dy).to("cuda", F32), both[offset:], V)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref = np.zeros((V, d), np.int64)
    np.add.at(ref, tok[tok >= 0], dy[tok >= 0])
    assert np.array_equal(dw.cpu().numpy().astype(np.int64), ref)


@pytest.mark.parametrize("T", [6, 600])
def test_tokens_outside_raise_and_are_read_as_none(T):
    rng = np.random.default_rng(4)
    V, d = 50, 40
    tok = _tokens(rng, T, V, "uniform")
    tok[1], tok[4] = V, -2
    tok[5] = 2 ** 31 - 1
    clean = np.where((tok < 0) | (tok >= V), -1, tok)
    w, dy = _rand(rng, (V, d), BF16), _rand(rng, (T, d), BF16)
    op = tw.Embedding(T, V, d)
    y = op.forward(_i32(tok), w)
    assert op.status.item() == _lib.TW_EINVAL
    assert (_f64(y) == ends.embedding(clean, _f64(w))).all()
    op.status.zero_()
    dw = op.backward(dy, _i32(tok))
    assert op.status.item() == _lib.TW_EINVAL
    _check_grad(dw, dy, clean, V, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,V,d", [(90, 40, 1), (90, 40, 3), (700, 40, 33), (600, 7, 257), (90, 40, 1027), (600, 9, 2050)])
def test_rows_at_any_offset_touch_their_own_columns_only(dtype, T, V, d):
    rng = np.random.default_rng(T + d)
    tok, lib = _tokens(rng, T, V, "zipf"), tw.load()
    dt = {F32: 0, BF16: 1, F16: 2}[dtype]
    op = tw.Embedding(T, V, d, dtype=dtype)
    t = _i32(tok)
    stream = torch.cuda.current_stream().cuda_stream

    def inside(rows, off, pad, fill, values, dt_):
        buf = torch.full((rows, off + d + pad), fill, dtype=dt_, device="cuda")
        if values is not None:
            buf[:, off:off + d] = values
        return buf, buf[:, off:off + d]

    w0, dy0, old = _rand(rng, (V, d), dtype), _rand(rng, (T, d), dtype), _rand(rng, (V, d), F32)
    for offs in ((0, 1, 2, 3), (1, 6, 0, 5), (7, 3, 4, 1), (8, 0, 6, 8)):
        (_, w), (yb, y) = inside(V, offs[0], offs[1] % 3, float("nan"), w0, dtype), inside(T, offs[1], offs[2] % 5, 9.0, None, dtype)
        assert lib.tw_embedding_fwd(t.data_ptr(), w.data_ptr(), w.stride(0), T, V, d, 1.0, dt, dt, y.data_ptr(), y.stride(0),
                                    op.status.data_ptr(), stream) == _lib.TW_OK
        assert (_f64(y) == ends.embedding(tok, _f64(w0))).all()
        assert (yb[:, :offs[1]] == 9).all() and (yb[:, offs[1] + d:] == 9).all()
        (_, dy) = inside(T, offs[2], offs[3] % 4, float("nan"), dy0, dtype)
        for add in (0, 1):
            wb, dw = inside(V, offs[3], offs[0] % 5, 9.0, old if add else None, F32)
            assert lib.tw_embedding_bwd(dy.data_ptr(), dy.stride(0), t.data_ptr(), T, V, d, 1.0, dt, add, dw.data_ptr(), dw.stride(0),
                                        op.ws.data_ptr(), op.ws_bytes, op.status.data_ptr(), stream) == _lib.TW_OK
            _check_grad(dw, dy0, tok, V, 1.0, old if add else None)
            assert (wb[:, :offs[3]] == 9).all() and (wb[:, offs[3] + d:] == 9).all()


def test_offsets_past_32_bits():
    """A table of over 2^31 elements: its last rows are read and written."""
    V, d = 140000, 16000
    w = torch.zeros((V, d), dtype=BF16, device="cuda")
    w[-1], w[0] = 2.0, 1.0
    op = tw.Embedding(4, V, d, dweight=False)
    tok = _i32([V - 1, 0, -1, V - 2])
    y = op.forward(tok, w)
    assert (y[0] == 2).all() and (y[1] == 1).all() and not y[2:].any()
    del w
    dw = torch.ones((V, d), device="cuda")
    op.backward(y.fill_(0.5), tok, out=dw, add=True)
    assert (dw[-2:] == 1.5).all() and (dw[0] == 1.5).all() and (dw[1:-2:997] == 1).all()
    many = torch.full((600,), V - 1, dtype=torch.int32, device="cuda")
    big = tw.Embedding(600, V, d, dweight=False)
    big.backward(torch.ones((600, d), dtype=BF16, device="cuda"), many, out=dw)
    assert (dw[-1] == 600).all() and not dw[:-1:1009].any() and not dw[-2].any()


def test_no_tokens():
    op = tw.Embedding(4, 6, 8)
    op.dweight.fill_(3)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dy = torch.empty((0, 8), dtype=BF16, device="cuda")
    assert (op.backward(dy, none, add=True) == 3).all()
    assert not op.backward(dy, none).any()
    assert op.forward(none, torch.ones((6, 8), dtype=BF16, device="cuda")).shape == (0, 8)


def test_shapes_of_tokens_and_a_side_stream():
    rng = np.random.default_rng(11)
    tok, w = _i32(rng.integers(0, 30, (4, 5))), _rand(rng, (30, 64), BF16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy = torch.zeros(1 << 26, device="cuda").add_(1)
        later = tok + 0
        op = tw.Embedding(20, 30, 64)
        y = op.forward(later, w)
        dw = op.backward(y, later)
    s.synchronize()
    assert torch.equal(y, w[tok.view(-1).long()]) and busy[0] == 1
    _check_grad(dw, y, tok.cpu().numpy().reshape(-1), 30, 1.0)
    y2, status = tw.embedding_fwd(tok, w, scale=2.0)
    assert status.item() == 0 and torch.equal(y2, 2 * y)


def test_captured_and_replayed():
    rng = np.random.default_rng(12)
    V, d, T = 64, 128, 700
    tok, w, dy = _i32(rng.integers(-1, V, T)), _rand(rng, (V, d), BF16), _rand(rng, (T, d), BF16)
    op = tw.Embedding(T, V, d)
    op.forward(tok, w), op.backward(dy, tok)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = op.forward(tok, w)
        dw = op.backward(dy, tok)
    for _ in range(3):
        tok.copy_(_i32(rng.integers(-1, V, T)))
        graph.replay()
        t = tok.cpu().numpy()
        assert (_f64(y) == ends.embedding(t, _f64(w))).all()
        _check_grad(dw, dy, t, V, 1.0)
