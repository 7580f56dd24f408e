"""Host-side refusals of the RMS norm, embedding and orthogonalised-update entry points: every
call here is rejected (or has no rows) before anything reaches a GPU. And of the binding, whose
operands here are stand-ins that say they are on a GPU."""
import ctypes
import math
import os

import pytest

import activation_sparse_feedforward_gb300 as tw
from activation_sparse_feedforward_gb300 import _lib, row_ops

torch = pytest.importorskip("torch")

P = 4096  # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()
    return tw.load()


def _rms_fwd(lib, **kw):
    a = dict(x=P, ldx=64, res=None, ldres=0, w=P, T=4, d=64, eps=1e-6, dtype=1, wtype=0, sum=None, ldsum=64, y=P, ldy=64, rstd=P)
    assert set(kw) <= set(a)
    return lib.tw_rms_norm_fwd(*{**a, **kw}.values(), None)


FWD = [
    (dict(T=-1), "EINVAL"), (dict(d=0), "EINVAL"), (dict(d=16385), "EUNSUPPORTED"), (dict(T=(1 << 30) + 1), "EUNSUPPORTED"),
    (dict(dtype=3), "EINVAL"), (dict(dtype=-1), "EINVAL"), (dict(wtype=2), "EINVAL"), (dict(eps=-1.0), "EINVAL"),
    (dict(eps=math.nan), "EINVAL"), (dict(eps=math.inf), "EINVAL"), (dict(x=None), "EINVAL"), (dict(x=P + 1), "EALIGN"),
    (dict(w=P + 2), "EALIGN"), (dict(ldx=-1), "EINVAL"), (dict(sum=P), "EINVAL"), (dict(res=P, ldres=64, sum=P, ldsum=8), "EINVAL"),
    (dict(rstd=P + 2), "EALIGN"),
]


@pytest.mark.parametrize("kw,code", FWD + [(dict(y=None), "EINVAL"), (dict(ldy=63), "EINVAL"), (dict(y=P + 1), "EALIGN"),
                                           (dict(T=0, x=None, y=None), "OK")], ids=str)
def test_rms_norm_fwd_refusals(lib, kw, code):
    assert _rms_fwd(lib, **kw) == getattr(_lib, "TW_" + code)


def _rms_fp8(lib, **kw):
    a = dict(x=P, ldx=64, res=None, ldres=0, w=P, T=4, d=64, eps=1e-6, dtype=1, wtype=0, sum=None, ldsum=64, q=P, ldq=64, scales=P,
             group=0, rstd=P)
    assert set(kw) <= set(a)
    return lib.tw_rms_norm_fwd_fp8(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", FWD + [
    (dict(q=None), "EINVAL"), (dict(ldq=63), "EINVAL"), (dict(scales=None), "EINVAL"), (dict(scales=P + 2), "EALIGN"),
    (dict(group=-1), "EINVAL"), (dict(group=64), "EUNSUPPORTED"), (dict(T=0, x=None, q=None, scales=None), "OK")], ids=str)
def test_rms_norm_fwd_fp8_refusals(lib, kw, code):
    assert _rms_fp8(lib, **kw) == getattr(_lib, "TW_" + code)


def _rms_bwd(lib, **kw):
    need = lib.tw_rms_norm_bwd_workspace_size(kw.get("T", 4), kw.get("d", 64))
    a = dict(dy=P, lddy=64, x=P, ldx=64, rstd=P, w=P, dres=None, lddres=0, T=4, d=64, dtype=1, wtype=0, dx=P, lddx=64, dw=P, ws=P,
             ws_bytes=need)
    assert set(kw) <= set(a)
    return lib.tw_rms_norm_bwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(d=20000), "EUNSUPPORTED"), (dict(dy=None), "EINVAL"), (dict(rstd=None), "EINVAL"),
    (dict(rstd=P + 1), "EALIGN"), (dict(lddx=10), "EINVAL"), (dict(dres=P + 1, lddres=64), "EALIGN"), (dict(dw=P + 2), "EALIGN"),
    (dict(ws=None), "EINVAL"), (dict(ws=P + 8), "EALIGN"), (dict(ws_bytes=255), "EWORKSPACE"),
    (dict(T=0, dw=None, dy=None, x=None, dx=None, rstd=None, ws=None), "OK"),
], ids=str)
def test_rms_norm_bwd_refusals(lib, kw, code):
    assert _rms_bwd(lib, **kw) == getattr(_lib, "TW_" + code)


def test_rms_norm_bwd_workspace(lib):
    size = lib.tw_rms_norm_bwd_workspace_size
    assert size(0, 64) == 0 and size(1, 64) >= 64 * 4 and size(1 << 20, 2048) == size(1 << 24, 2048)


def _embed_fwd(lib, **kw):
    a = dict(tokens=P, w=P, ldw=64, T=4, V=10, d=64, scale=1.0, dtype=1, wtype=1, y=P, ldy=64, status=P)
    assert set(kw) <= set(a)
    return lib.tw_embedding_fwd(*{**a, **kw}.values(), None)


SIZES = [(dict(T=-1), "EINVAL"), (dict(V=0), "EINVAL"), (dict(d=0), "EINVAL"), (dict(d=16385), "EUNSUPPORTED"),
         (dict(T=(1 << 22) + 1), "EUNSUPPORTED"), (dict(V=(1 << 22) + 1), "EUNSUPPORTED"), (dict(scale=math.nan), "EINVAL"),
         (dict(scale=math.inf), "EINVAL"), (dict(dtype=3), "EINVAL"), (dict(tokens=None), "EINVAL"), (dict(tokens=P + 2), "EALIGN"),
         (dict(status=None), "EINVAL")]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(wtype=2), "EINVAL"), (dict(w=None), "EINVAL"), (dict(ldw=-1), "EINVAL"), (dict(ldy=63), "EINVAL"), (dict(y=P + 1), "EALIGN"),
    (dict(wtype=0, w=P + 2), "EALIGN"), (dict(T=0, tokens=None, w=None, y=None), "OK")], ids=str)
def test_embedding_fwd_refusals(lib, kw, code):
    assert _embed_fwd(lib, **kw) == getattr(_lib, "TW_" + code)


def _embed_bwd(lib, **kw):
    need = lib.tw_embedding_bwd_workspace_size(kw.get("T", 600), kw.get("V", 10), kw.get("d", 64))
    a = dict(dy=P, lddy=64, tokens=P, T=600, V=10, d=64, scale=1.0, dtype=1, add=0, dw=P, lddw=64, ws=P, ws_bytes=need, status=P)
    assert set(kw) <= set(a)
    return lib.tw_embedding_bwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dy=None), "EINVAL"), (dict(lddy=-1), "EINVAL"), (dict(dw=None), "EINVAL"), (dict(lddw=63), "EINVAL"), (dict(dw=P + 2), "EALIGN"),
    (dict(ws=None), "EINVAL"), (dict(ws=P + 8), "EALIGN"), (dict(ws_bytes=1000), "EWORKSPACE"),
    (dict(T=0, add=1, dy=None, tokens=None, ws=None), "OK")], ids=str)
def test_embedding_bwd_refusals(lib, kw, code):
    assert _embed_bwd(lib, **kw) == getattr(_lib, "TW_" + code)


def test_embedding_workspace(lib):
    size = lib.tw_embedding_bwd_workspace_size
    assert size(512, 1000, 64) == 0 and size(513, 1000, 64) >= 513 * 8 and size(-1, 10, 10) == 0
    # four words a token, and for long batches no more parts of runs than 6000 chunks have
    assert size(1 << 22, 1000, 64) < (1 << 22) * 16 + 2 * 4 * 256 * 6010 + 10000


def _pointers(*values):
    return (ctypes.c_void_p * len(values))(*values)


BIG = 1 << 40  # far between the fake matrices


def _ortho(lib, **kw):
    coef = kw.pop("coef_values", [3.4445, -4.775, 2.0315] * 5)
    m, n, count = kw.get("m", 64), kw.get("n", 64), kw.get("count", 1)
    at = lambda k: _pointers(*[(k + 3 * i) * BIG for i in range(max(count, 1))])  # noqa: E731
    a = dict(grads=at(1), ldg=64, gtype=0, buffers=at(2), ldb=64, mu=0.9, nesterov=1,
             count=count, m=m, n=n, steps=5, coef=(ctypes.c_float * len(coef))(*coef), scale=1.0, beta=0.0,
             out=at(3), ldo=64, otype=1, ws=P,
             ws_bytes=lib.tw_orthogonalize_workspace_size(m, n, count), status=P)
    assert set(kw) <= set(a)
    return lib.tw_orthogonalize(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(m=0), "EINVAL"), (dict(n=-1), "EINVAL"), (dict(count=0), "EINVAL"), (dict(count=9), "EUNSUPPORTED"),
    (dict(m=16385, n=16385), "EUNSUPPORTED"), (dict(m=(1 << 20) + 1), "EUNSUPPORTED"), (dict(gtype=3), "EINVAL"), (dict(otype=-1), "EINVAL"),
    (dict(grads=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(coef=None), "EINVAL"), (dict(steps=0), "EINVAL"),
    (dict(steps=33, coef_values=[1.0] * 99), "EINVAL"), (dict(mu=math.nan), "EINVAL"), (dict(scale=math.inf), "EINVAL"),
    (dict(beta=math.nan), "EINVAL"), (dict(coef_values=[1.0] * 14 + [math.inf]), "EINVAL"), (dict(grads=_pointers(None)), "EINVAL"),
    (dict(grads=_pointers(P + 2)), "EALIGN"), (dict(ldg=63), "EINVAL"), (dict(buffers=_pointers(None)), "EINVAL"),
    (dict(buffers=_pointers(P + 2)), "EALIGN"), (dict(ldb=63), "EINVAL"), (dict(out=_pointers(None)), "EINVAL"),
    (dict(out=_pointers(P + 1)), "EALIGN"), (dict(ldo=63), "EINVAL"), (dict(ws=None), "EINVAL"), (dict(ws=P + 8), "EALIGN"),
    (dict(ws_bytes=10), "EWORKSPACE"), (dict(status=None), "EINVAL"), (dict(status=P + 2), "EALIGN"),
], ids=str)
def test_orthogonalize_refusals(lib, kw, code):
    assert _ortho(lib, **kw) == getattr(_lib, "TW_" + code)


def test_orthogonalize_shared_memory(lib):
    """Matrices that are written and share an element are refused; the library goes on to the
    workspace's size (here too small) where they do not."""
    ok, bad = _lib.TW_EWORKSPACE, _lib.TW_EINVAL
    m, n, row = 64, 64, 200  # rows of 200 elements: room for three matrices side by side

    def out(*offsets, size=2, **kw):
        return _ortho(lib, count=2, ldo=row, ws_bytes=1, out=_pointers(*[7 * BIG + size * o for o in offsets]), **kw)

    assert out(0, m * row) == ok and out(0, 64) == ok and out(136, 64) == ok      # below, beside, beside
    assert out(0, 0) == bad and out(0, 63) == bad and out(0, 64 * row - 137) == bad
    assert out(0, row - 63) == bad                                                # its columns wrap into the next row's first
    assert out(0, (m - 1) * row + 64) == ok and out(0, (m - 1) * row + 63) == bad  # behind the last row
    assert out(0, 64, size=4, otype=0) == ok and out(0, 63, size=4, otype=0) == bad
    same = _pointers(BIG, BIG)
    assert _ortho(lib, count=2, buffers=same) == bad
    assert _ortho(lib, count=2, buffers=_pointers(5 * BIG, 5 * BIG + 4 * 64 * 64), ws_bytes=1) == ok
    assert _ortho(lib, count=2, grads=same, buffers=None, ws_bytes=1) == ok        # read alone
    assert _ortho(lib, buffers=_pointers(BIG)) == bad                              # a buffer in its gradient
    assert _ortho(lib, buffers=_pointers(BIG + 4 * 64 * 64), ws_bytes=1) == ok
    assert _ortho(lib, gtype=1, buffers=_pointers(BIG + 64 * 64)) == bad           # two bytes an element and four
    assert _ortho(lib, out=_pointers(BIG), otype=0, ws_bytes=1) == ok              # the result in the gradient's place


def test_orthogonalize_workspace(lib):
    size = lib.tw_orthogonalize_workspace_size
    assert size(0, 4, 1) == 0 and size(4, 4, 9) == 0
    assert size(5632, 2048, 3) >= 3 * 3 * 5632 * 2048 * 2 and size(2048, 5632, 3) == size(5632, 2048, 3)


def test_workspace_serves_smaller_calls(lib):
    """A workspace made for so many tokens or matrices has room for fewer: fewer tokens may go
    in smaller chunks, fewer matrices in more slices."""
    size = lib.tw_embedding_bwd_workspace_size
    tokens = [512, 513, 4096, 4799, 4800, 4803, 4804, 9599, 9600, 9607, 9608, 24000, 24004, 65535, 65536, 65551, 65552, 70000, 131000, 131103, 131104, 262207, 262208, 1 << 22]
    for d in (64, 1027, 8192):
        sizes = [size(t, 5003, d) for t in tokens]
        assert sizes == sorted(sizes)
    for m in list(range(64, 4200, 448)) + [1, 3712, 3904]:
        for n in list(range(64, 4200, 448)) + [1, 448]:
            sizes = [lib.tw_orthogonalize_workspace_size(m, n, k) for k in range(1, 9)]
            assert sizes == sorted(sizes), (m, n)


# ------------------------------------------------------------------------------ the binding

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""

    @staticmethod
    def of(t, index=0):
        t = t.as_subclass(OnGpu)
        t.index_ = index
        return t

    def get_device(self):
        return getattr(self, "index_", 0)


class Notes:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def current_device(monkeypatch):
    at = [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return at


def _at(op, notes, index=0):
    op._lib, op._device, op._stream = notes, index, row_ops._stream_of(index)
    return op


T, D, V = 4, 8, 6
MATRIX, VECTOR = ((T, D), BF16), ((T,), F32)
CALLS = {
    "rms_fwd": (lambda: tw.RMSNorm(T, D, device="cpu"), lambda op, a: op.forward(a["x"], a["weight"], residual=a["residual"]),
                dict(x=MATRIX, weight=((D,), BF16), residual=MATRIX)),
    "rms_fp8": (lambda: tw.RMSNorm(T, D, fp8=True, device="cpu"),
                lambda op, a: op.forward_fp8(a["x"], a["weight"], residual=a["residual"]),
                dict(x=MATRIX, weight=((D,), BF16), residual=MATRIX)),
    "rms_bwd": (lambda: tw.RMSNorm(T, D, device="cpu"),
                lambda op, a: op.backward(a["dy"], a["x"], a["weight"], a["dres"], a["rstd"]),
                dict(dy=MATRIX, x=MATRIX, weight=((D,), BF16), dres=MATRIX, rstd=VECTOR)),
    "embed_fwd": (lambda: tw.Embedding(T, V, D, device="cpu"), lambda op, a: op.forward(a["tokens"], a["weight"]),
                  dict(tokens=((T,), I32), weight=((V, D), BF16))),
    "embed_bwd": (lambda: tw.Embedding(T, V, D, device="cpu"), lambda op, a: op.backward(a["dy"], a["tokens"], out=a["out"], add=True),
                  dict(dy=MATRIX, tokens=((T,), I32), out=((V, D), F32))),
    "ortho": (lambda: tw.Orthogonalize(T, D, device="cpu"), lambda op, a: op(a["grads"], a["buffers"], out=a["out"], beta=0.5),
              dict(grads=((T, D), F32), buffers=((T, D), F32), out=MATRIX)),
}


def _operands(which, index=0, **other):
    return {k: OnGpu.of(torch.zeros(shape, dtype=dtype), other.get(k, index)) for k, (shape, dtype) in CALLS[which][2].items()}


@pytest.mark.parametrize("which", CALLS)
def test_operands_on_the_objects_device_reach_the_library(lib, which, current_device):
    for index in (0, 1):
        current_device[0] = index
        notes = Notes()
        CALLS[which][1](_at(CALLS[which][0](), notes, index), _operands(which, index))
        assert len(notes.calls) == 1


@pytest.mark.parametrize("which,operand", [(w, o) for w in CALLS for o in CALLS[w][2]])
def test_an_operand_on_another_device_or_of_another_type_is_refused(lib, which, operand, current_device):
    notes = Notes()
    op = _at(CALLS[which][0](), notes)
    with pytest.raises(ValueError, match=f"{operand}.* must be .*device"):
        CALLS[which][1](op, _operands(which, 0, **{operand: 1}))
    a = _operands(which)
    a[operand] = OnGpu.of(torch.zeros(a[operand].shape, dtype=torch.float64))
    with pytest.raises(ValueError, match=f"{operand}.* must be "):
        CALLS[which][1](op, a)
    assert not notes.calls


@pytest.mark.parametrize("which", CALLS)
def test_another_current_device_and_host_buffers_are_refused(lib, which, current_device):
    notes = Notes()
    current_device[0] = 1
    with pytest.raises(ValueError, match="current device"):
        CALLS[which][1](_at(CALLS[which][0](), notes), _operands(which))
    current_device[0] = 0
    op = CALLS[which][0]()
    op._lib = notes
    with pytest.raises(ValueError, match="CUDA"):
        CALLS[which][1](op, _operands(which))
    assert not notes.calls


def test_what_an_object_was_not_made_for_is_refused(lib, current_device):
    notes = Notes()
    with pytest.raises(ValueError, match="weight_dtype"):
        tw.RMSNorm(4, 8, weight_dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="group"):
        tw.RMSNorm(4, 8, fp8=True, group=64, device="cpu")
    with pytest.raises(ValueError, match="backward=False"):
        tw.RMSNorm(4, 8, backward=False, device="cpu").backward(None, None)
    a = _operands("rms_fwd")
    with pytest.raises(ValueError, match="forward_fp8"):
        _at(tw.RMSNorm(T, D, fp8=True, device="cpu"), notes).forward(a["x"])
    with pytest.raises(ValueError, match="fp8=False"):
        _at(tw.RMSNorm(T, D, device="cpu"), notes).forward_fp8(a["x"])
    with pytest.raises(ValueError, match="at most 3 rows"):
        _at(tw.RMSNorm(3, D, device="cpu"), notes).forward(a["x"])
    e = _operands("embed_bwd")
    with pytest.raises(ValueError, match="backward=False"):
        _at(tw.Embedding(T, V, D, backward=False, device="cpu"), notes).backward(e["dy"], e["tokens"])
    with pytest.raises(ValueError, match="dweight=False"):
        _at(tw.Embedding(T, V, D, dweight=False, device="cpu"), notes).backward(e["dy"], e["tokens"])
    with pytest.raises(ValueError, match="at most 3"):
        _at(tw.Embedding(3, V, D, device="cpu"), notes).backward(e["dy"], e["tokens"])
    with pytest.raises(ValueError, match="dy has shape"):
        _at(tw.Embedding(T, V, D, device="cpu"), notes).backward(e["dy"], e["tokens"][:3])
    assert not notes.calls


def test_orthogonalize_lists(lib, current_device):
    notes, g = Notes(), OnGpu.of(torch.zeros(4, 8))
    for kw in (dict(m=0), dict(count=9), dict(steps=0), dict(steps=33), dict(coefficients=(1.0, 2.0)), dict(coefficients=[(1, 2, 3)] * 4),
               dict(dtype=torch.float64), dict(n=20000, m=20000)):
        with pytest.raises(ValueError):
            tw.Orthogonalize(**{**dict(m=4, n=8, device="cpu"), **kw})
    op = _at(tw.Orthogonalize(4, 8, count=2, device="cpu"), notes)
    with pytest.raises(ValueError, match="momentum 0"):
        op([g])
    with pytest.raises(ValueError, match="1 to 2 matrices"):
        op([g] * 3, [g] * 3)
    with pytest.raises(ValueError, match="1 to 2 matrices"):
        op([], [])
    with pytest.raises(ValueError, match="buffers has 1"):
        op([g, g], [g])
    with pytest.raises(ValueError, match="needs `out`"):
        op([g], [g], beta=1.0)
    wide = OnGpu.of(torch.zeros(4, 16)[:, :8])
    with pytest.raises(ValueError, match="one row stride"):
        op([g, wide], [g, g])
    with pytest.raises(ValueError, match="overlapping"):
        op([OnGpu.of(torch.zeros(1, 8).expand(4, 8))], [g])
    with pytest.raises(ValueError, match="shape"):
        op([g.T], [g])
    assert not notes.calls
    assert len(op([g], [g])) == 1 and isinstance(op(g, g), torch.Tensor)  # (the library here only takes notes)
    assert [c[0] for c in notes.calls] == ["tw_orthogonalize"] * 2
