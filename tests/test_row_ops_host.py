"""Host-side refusals of the layer norm, distillation and log-probability entry points:
every call here is rejected (or has no rows) before anything reaches a GPU."""
import ctypes
import math
import os

import pytest

import activation_sparse_feedforward_gb300 as tw
from activation_sparse_feedforward_gb300 import _lib

torch = pytest.importorskip("torch")

P = 4096  # fake, aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()
    return tw.load()


def _norm_fwd(lib, **kw):
    a = dict(x=P, ldx=64, res=None, ldres=0, w=P, b=P, T=4, d=64, eps=1e-5, dtype=1, wtype=0, sum=None, ldsum=64, y=P,
             ldy=64, mean=P, rstd=P)
    assert set(kw) <= set(a)
    return lib.tw_layer_norm_fwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(d=0), "EINVAL"), (dict(d=16385), "EUNSUPPORTED"),
    (dict(T=(1 << 30) + 1), "EUNSUPPORTED"), (dict(dtype=3), "EINVAL"),
    (dict(dtype=-1), "EINVAL"), (dict(wtype=2), "EINVAL"), (dict(eps=-1.0), "EINVAL"), (dict(eps=math.nan), "EINVAL"),
    (dict(eps=math.inf), "EINVAL"), (dict(x=None), "EINVAL"), (dict(y=None), "EINVAL"), (dict(x=P + 1), "EALIGN"),
    (dict(w=P + 2), "EALIGN"), (dict(ldy=63), "EINVAL"), (dict(ldx=-1), "EINVAL"), (dict(sum=P), "EINVAL"),
    (dict(res=P, ldres=64, sum=P, ldsum=8), "EINVAL"), (dict(mean=P + 2), "EALIGN"), (dict(T=0, x=None, y=None), "OK"),
], ids=str)
def test_layer_norm_fwd_refusals(lib, kw, code):
    assert _norm_fwd(lib, **kw) == getattr(_lib, "TW_" + code)


def _norm_bwd(lib, **kw):
    need = lib.tw_layer_norm_bwd_workspace_size(kw.get("T", 4), kw.get("d", 64))
    a = dict(dy=P, lddy=64, x=P, ldx=64, mean=P, rstd=P, w=P, dres=None, lddres=0, T=4, d=64, dtype=1, wtype=0, dx=P,
             lddx=64, dw=P, db=P, ws=P, ws_bytes=need)
    assert set(kw) <= set(a)
    return lib.tw_layer_norm_bwd(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "EINVAL"), (dict(d=20000), "EUNSUPPORTED"), (dict(dy=None), "EINVAL"), (dict(mean=None), "EINVAL"),
    (dict(rstd=P + 1), "EALIGN"), (dict(lddx=10), "EINVAL"), (dict(dres=P + 1, lddres=64), "EALIGN"),
    (dict(dw=P + 2), "EALIGN"), (dict(ws=None), "EINVAL"), (dict(ws=P + 8), "EALIGN"), (dict(ws_bytes=511), "EWORKSPACE"),
    (dict(T=0, dw=None, db=None, dy=None, x=None, dx=None, mean=None, rstd=None, ws=None), "OK"),
], ids=str)
def test_layer_norm_bwd_refusals(lib, kw, code):
    assert _norm_bwd(lib, **kw) == getattr(_lib, "TW_" + code)


def test_layer_norm_bwd_workspace(lib):
    size = lib.tw_layer_norm_bwd_workspace_size
    assert size(0, 64) == 0 and size(1, 64) >= 2 * 64 * 4
    assert size(1 << 20, 2048) == size(1 << 24, 2048)  # bounded whatever the number of rows


def _distill(lib, **kw):
    a = dict(z=P, ldz=100, N=4, V=100, dtype=1, idx=P, val=P, vtype=0, K=8, rest=None, labels=None, tau=1.0, kd=1.0,
             ce=0.0, dloss=None, scale=1.0, loss=P, dz=P, lddz=100, status=P)
    assert set(kw) <= set(a)
    return lib.tw_distill(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), "EINVAL"), (dict(V=0), "EINVAL"), (dict(V=393217, ldz=400000, lddz=400000), "EUNSUPPORTED"),
    (dict(N=(1 << 27) + 1), "EUNSUPPORTED"), (dict(dtype=9), "EINVAL"), (dict(vtype=-1), "EINVAL"), (dict(K=-1), "EINVAL"),
    (dict(K=1025), "EUNSUPPORTED"), (dict(tau=0.0), "EINVAL"), (dict(tau=-1.0), "EINVAL"), (dict(tau=math.nan), "EINVAL"), (dict(tau=1e-7), "EINVAL"),
    (dict(tau=2e6), "EINVAL"),
    (dict(tau=math.inf), "EINVAL"), (dict(kd=math.nan), "EINVAL"), (dict(scale=math.inf), "EINVAL"),
    (dict(loss=None, dz=None), "EINVAL"), (dict(z=None), "EINVAL"), (dict(z=P + 1), "EALIGN"), (dict(lddz=99), "EINVAL"),
    (dict(ldz=-5), "EINVAL"), (dict(idx=None), "EINVAL"), (dict(val=None), "EINVAL"), (dict(val=P + 2), "EALIGN"),
    (dict(idx=P + 2), "EALIGN"), (dict(rest=P + 1), "EALIGN"), (dict(status=None), "EINVAL"),
    (dict(ce=1.0, labels=P + 1), "EALIGN"), (dict(N=0, z=None, dz=None), "OK"),
], ids=str)
def test_distill_refusals(lib, kw, code):
    assert _distill(lib, **kw) == getattr(_lib, "TW_" + code)


def _logprobs(lib, **kw):
    a = dict(z=P, ldz=100, N=4, V=100, dtype=1, tokens=P, S=1, tau=1.0, K=4, logprob=P, entropy=P, idx=P, top=P, status=P)
    assert set(kw) <= set(a)
    return lib.tw_token_logprobs(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), "EINVAL"), (dict(V=0), "EINVAL"), (dict(V=393217), "EUNSUPPORTED"), (dict(S=-1), "EINVAL"),
    (dict(K=-1), "EINVAL"), (dict(K=129), "EUNSUPPORTED"), (dict(tau=0.0), "EINVAL"), (dict(tokens=None), "EINVAL"),
    (dict(logprob=None), "EINVAL"), (dict(idx=None), "EINVAL"), (dict(top=P + 2), "EALIGN"), (dict(entropy=P + 1), "EALIGN"),
    (dict(z=P + 1), "EALIGN"), (dict(status=None), "EINVAL"), (dict(N=0, z=None), "OK"),
], ids=str)
def test_token_logprobs_refusals(lib, kw, code):
    assert _logprobs(lib, **kw) == getattr(_lib, "TW_" + code)


def test_python_binding_refuses_host_tensors_and_wrong_shapes(lib):
    ln = tw.LayerNorm(4, 8, device="cpu")  # buffers only: no call reaches the library
    with pytest.raises(ValueError, match="CUDA"):
        ln.forward(torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="at most 4 rows"):
        ln.forward(torch.zeros(5, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="weight_dtype"):
        tw.LayerNorm(4, 8, dtype=torch.bfloat16, weight_dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="dtype must be"):
        tw.DistillLoss(4, 8, 2, dtype=torch.float64, device="cpu")
    with pytest.raises(ValueError, match="backward=False"):
        tw.LayerNorm(4, 8, backward=False, device="cpu").backward(None, None)
    with pytest.raises(ValueError, match="CUDA"):
        tw.TokenLogprobs(4, 8, device="cpu")(torch.zeros(4, 8, dtype=torch.bfloat16))
