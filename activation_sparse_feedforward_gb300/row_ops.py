"""Torch-facing binding of the operators at the ends of a model around the feedforward
layer: layer norm, the distillation loss and token log probabilities (see the last
part of include/twell.h).

As in ``ops``: objects preallocate every buffer, calls enqueue on torch's current
stream and neither allocate nor synchronise; one-shot functions build such an object.
Matrices are [rows, columns] views with unit column stride and any row stride; a call
may pass fewer rows than the object was made for and gets views of that many rows back.
Every operand is on the object's device, and that is the current one; else ValueError.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from .ops import _workspace

DTYPES = {torch.float32: _lib.TW_F32, torch.bfloat16: _lib.TW_BF16, torch.float16: _lib.TW_F16}


def _dtype_code(dtype: torch.dtype) -> int:
    code = DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    return code


def _matrix(name: str, t: torch.Tensor, dtype: torch.dtype, device: int, rows: int, cols: int) -> int:
    """Checks a [rows, cols] matrix; its row stride in elements (a single row's is its
    length, whatever torch says). device: see _device_of."""
    if t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA {dtype} tensor on the object's device")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.is_contiguous():
        return cols
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return ld if rows > 1 else cols


def _vector(name: str, t: torch.Tensor | None, dtype: torch.dtype, device: int, n: int) -> int | None:
    """Checks a contiguous side array of n elements, or None; its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != device or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of {n} elements on the object's device")
    return t.data_ptr()


def _list(name: str, t: torch.Tensor, dtype: torch.dtype, device: int, n: int, k: int) -> int:
    """Checks a contiguous array of n rows of k entries (the entries last, or all in one
    dimension); its address."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor on the object's device")
    if t.shape != (n, k) and (t.numel() != n * k or not (k == 1 or t.dim() == 1 or t.shape[-1] == k)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, k)}")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, most: int) -> int:
    if t.dim() != 2 or (n := t.shape[0]) > most:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected at most {most} rows")
    return n


def _addresses(*buffers: torch.Tensor | None) -> tuple[int | None, ...]:
    """An object's own buffers' addresses, asked for once."""
    return tuple(None if t is None else t.data_ptr() for t in buffers)


def _device_of(buffer: torch.Tensor) -> int:
    """The index of an object's GPU; where its buffers are on the host, one that no tensor has."""
    index = buffer.get_device()
    return index if index >= 0 else -2


def _stream_of(device: int):
    """What gives the device's raw current stream: torch.cuda.current_stream() builds a Stream
    object for it, 2.9 us of a small call's host time against 0.1. A launch goes to the current
    device, so with several GPUs that has to be this one."""
    if torch.cuda.device_count() == 1:
        return functools.partial(torch._C._cuda_getCurrentRawStream, device)

    def checked() -> int:
        if torch._C._cuda_getDevice() != device:
            raise ValueError(f"the operands are on cuda:{device}, which is not the current device")
        return torch._C._cuda_getCurrentRawStream(device)

    return checked


class LayerNorm:
    """Preallocated layer norm of up to T rows of width d, forward and backward (see
    tw_layer_norm_fwd, tw_layer_norm_bwd).

    weight_dtype: the type of weight and bias, `dtype` (default) or float32. backward:
    whether the buffers of the backward (dx, fp32 dweight and dbias, workspace) are kept.
    """

    def __init__(self, T: int, d: int, dtype: torch.dtype = torch.bfloat16, weight_dtype: torch.dtype | None = None,
                 eps: float = 1e-5, backward: bool = True, device="cuda"):
        self.T, self.d, self.dtype, self.eps = T, d, dtype, float(eps)
        self.weight_dtype = weight_dtype or dtype
        self._dt, self._wdt = _dtype_code(dtype), _dtype_code(self.weight_dtype)
        if self._wdt not in (self._dt, _lib.TW_F32):
            raise ValueError(f"weight_dtype must be {dtype} or float32, got {self.weight_dtype}")
        self._lib = _lib.load()
        self.y = torch.empty((T, d), dtype=dtype, device=device)
        self.sum = torch.empty((T, d), dtype=dtype, device=device)
        self._mean = torch.empty(T, dtype=torch.float32, device=device)
        self._rstd = torch.empty(T, dtype=torch.float32, device=device)
        #: fp32 row means, and 1 / sqrt(variance + eps), of the last forward's rows
        self.mean, self.rstd = self._mean, self._rstd
        self.dx = self.dweight = self.dbias = None
        if backward:
            self.dx = torch.empty((T, d), dtype=dtype, device=device)
            self.dweight = torch.empty(d, dtype=torch.float32, device=device)
            self.dbias = torch.empty(d, dtype=torch.float32, device=device)
            self.ws_bytes = int(self._lib.tw_layer_norm_bwd_workspace_size(T, d))
            self.ws = _workspace(self.ws_bytes, device)
            self._to_bwd = _addresses(self.dx, self.dweight, self.dbias, self.ws)
        self._to_fwd = _addresses(self.y, self.sum, self._mean, self._rstd)
        self._device = _device_of(self.y)
        self._stream = _stream_of(self._device)

    def forward(self, x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                residual: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """(y, s): s = x + residual (x itself without one), y = norm(s) weight + bias."""
        n, d, dt, dev = _rows("x", x, self.T), self.d, self.dtype, self._device
        ldx = _matrix("x", x, dt, dev, n, d)
        w, b = _vector("weight", weight, self.weight_dtype, dev, d), _vector("bias", bias, self.weight_dtype, dev, d)
        y, s = self.y, self.sum
        if n != self.T:
            y, s = y[:n], s[:n]
        if n != self.mean.shape[0]:
            self.mean, self.rstd = self._mean[:n], self._rstd[:n]
        to_y, to, to_mean, to_rstd = self._to_fwd
        if residual is None:
            r, ldr, to = None, 0, None
        else:
            r, ldr = residual.data_ptr(), _matrix("residual", residual, dt, dev, n, d)
        code = self._lib.tw_layer_norm_fwd(x.data_ptr(), ldx, r, ldr, w, b, n, d, self.eps, self._dt, self._wdt, to, d,
                                           to_y, d, to_mean, to_rstd, self._stream())
        if code:
            _lib.check(code, "tw_layer_norm_fwd")
        return y, (x if residual is None else s)

    def backward(self, dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None = None,
                 dres: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                 rstd: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(dx, dweight, dbias) for x the tensor that was normalised (the forward's s);
        dres is added to dx. mean, rstd: the statistics, of the last forward by default."""
        dx = self.dx
        if dx is None:
            raise ValueError("this LayerNorm was made with backward=False")
        n, d, dt, dev = _rows("x", x, self.T), self.d, self.dtype, self._device
        ldx, lddy = _matrix("x", x, dt, dev, n, d), _matrix("dy", dy, dt, dev, n, d)
        w = _vector("weight", weight, self.weight_dtype, dev, d)
        m = _vector("mean", self.mean if mean is None else mean, torch.float32, dev, n)
        r = _vector("rstd", self.rstd if rstd is None else rstd, torch.float32, dev, n)
        g, ldg = (None, 0) if dres is None else (dres.data_ptr(), _matrix("dres", dres, dt, dev, n, d))
        if n != self.T:
            dx = dx[:n]
        to, to_w, to_b, ws = self._to_bwd
        code = self._lib.tw_layer_norm_bwd(dy.data_ptr(), lddy, x.data_ptr(), ldx, m, r, w, g, ldg, n, d, self._dt,
                                           self._wdt, to, d, to_w, to_b, ws, self.ws_bytes, self._stream())
        if code:
            _lib.check(code, "tw_layer_norm_bwd")
        return dx, self.dweight, self.dbias


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, residual=None):
    """One-shot forward. Returns (y, s, mean, rstd)."""
    ln = LayerNorm(x.shape[0], x.shape[1], x.dtype, None if weight is None else weight.dtype, eps, backward=False,
                   device=x.device)
    y, s = ln.forward(x, weight, bias, residual)
    return y, s, ln.mean, ln.rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, dres=None):
    """One-shot backward. Returns (dx, dweight, dbias)."""
    ln = LayerNorm(x.shape[0], x.shape[1], x.dtype, None if weight is None else weight.dtype, device=x.device)
    return ln.backward(dy, x, weight, dres, mean, rstd)


class DistillLoss:
    """Preallocated distillation loss of up to N rows of V logits from a teacher's top K
    (see tw_distill): kd_weight * KD at `temperature` + ce_weight * cross entropy of the
    labels. K = 0 is plain cross entropy. grad: whether a gradient buffer dz is kept
    (calls may also name theirs with `out`, the logits themselves among them). A part whose
    weight is 0 is not looked at.

    idx [n, K] int32 (-1: no entry), val [n, K] float32, bfloat16 or float16, rest [n]
    float32 or None, labels [n] int32 (-1: none) or None. An index outside [-1, V)
    raises TW_EINVAL in `status`.
    """

    def __init__(self, N: int, V: int, K: int, dtype: torch.dtype = torch.bfloat16, temperature: float = 1.0,
                 kd_weight: float = 1.0, ce_weight: float = 0.0, grad: bool = True, device="cuda"):
        self.N, self.V, self.K, self.dtype = N, V, K, dtype
        self.temperature, self.kd_weight, self.ce_weight = float(temperature), float(kd_weight), float(ce_weight)
        self._dt = _dtype_code(dtype)
        self._lib = _lib.load()
        self.loss = torch.empty(N, dtype=torch.float32, device=device)
        self.dz = torch.empty((N, V), dtype=dtype, device=device) if grad else None
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._to = _addresses(self.loss, self.dz, self.status)
        self._device = _device_of(self.loss)
        self._stream = _stream_of(self._device)

    def _run(self, z, idx, val, rest, labels, dloss, scale, want_loss, want_grad, out):
        n, K, V, dev = _rows("z", z, self.N), self.K, self.V, self._device
        ld = _matrix("z", z, self.dtype, dev, n, V)
        to_loss, to_dz, status = self._to
        dz, to, ldd = None, None, 0
        if want_grad:
            dz = self.dz if out is None else out
            if dz is None:
                raise ValueError("this DistillLoss was made with grad=False: give `out`")
            if out is not None:
                to, ldd = out.data_ptr(), _matrix("out", out, self.dtype, dev, n, V)
            else:
                to, ldd = to_dz, V
                if n != self.N:
                    dz = dz[:n]
        i = v = None
        tdt = self._dt
        if K > 0 and self.kd_weight != 0.0:
            if idx is None or val is None:
                raise ValueError("idx and val must be given for K > 0")
            tdt = _dtype_code(val.dtype)
            i, v = _list("idx", idx, torch.int32, dev, n, K), _list("val", val, val.dtype, dev, n, K)
        r = None if rest is None else _vector("rest", rest, torch.float32, dev, n)
        lab = None if labels is None else _vector("labels", labels, torch.int32, dev, n)
        up = None if dloss is None else _vector("dloss", dloss, torch.float32, dev, n)
        code = self._lib.tw_distill(
            z.data_ptr(), ld, n, V, self._dt, i, v, tdt, K, r, lab, self.temperature, self.kd_weight, self.ce_weight, up,
            scale, to_loss if want_loss else None, to, ldd, status, self._stream())
        if code:
            _lib.check(code, "tw_distill")
        return (self.loss if n == self.N else self.loss[:n]), dz

    def forward(self, z, idx=None, val=None, rest=None, labels=None) -> torch.Tensor:
        """fp32 losses [n]."""
        return self._run(z, idx, val, rest, labels, None, 1.0, True, False, None)[0]

    def backward(self, z, idx=None, val=None, rest=None, labels=None, dloss=None, scale: float = 1.0,
                 out: torch.Tensor | None = None) -> torch.Tensor:
        """dz [n, V] = scale * dloss * d loss / d z (dloss [n] float32, None for 1)."""
        return self._run(z, idx, val, rest, labels, dloss, scale, False, True, out)[1]

    def forward_backward(self, z, idx=None, val=None, rest=None, labels=None, dloss=None, scale: float = 1.0,
                         out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """(losses, dz) in one pass over z."""
        return self._run(z, idx, val, rest, labels, dloss, scale, True, True, out)


def distill_loss(z, idx=None, val=None, rest=None, labels=None, temperature: float = 1.0, kd_weight: float = 1.0,
                 ce_weight: float = 0.0, dloss=None, scale: float = 1.0):
    """One-shot loss and gradient. Returns (losses, dz, status)."""
    op = DistillLoss(z.shape[0], z.shape[1], 0 if idx is None else idx.shape[1], z.dtype, temperature, kd_weight,
                     ce_weight, device=z.device)
    loss, dz = op.forward_backward(z, idx, val, rest, labels, dloss, scale)
    return loss, dz, op.status


class TokenLogprobs:
    """Preallocated log probabilities of n_tokens given tokens a row, with the entropy and
    the top_k alternatives of up to N rows of V logits (see tw_token_logprobs). A token
    outside [-1, V) raises TW_EINVAL in `status`."""

    def __init__(self, N: int, V: int, n_tokens: int = 1, top_k: int = 0, temperature: float = 1.0,
                 dtype: torch.dtype = torch.bfloat16, device="cuda"):
        self.N, self.V, self.n_tokens, self.top_k, self.dtype = N, V, n_tokens, top_k, dtype
        self.temperature = float(temperature)
        self._dt = _dtype_code(dtype)
        self._lib = _lib.load()
        self.logprob = torch.empty((N, n_tokens), dtype=torch.float32, device=device)
        self.entropy = torch.empty(N, dtype=torch.float32, device=device)
        self.top_idx = torch.empty((N, top_k), dtype=torch.int32, device=device)
        self.top_logprob = torch.empty((N, top_k), dtype=torch.float32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._to = _addresses(self.logprob, self.entropy, self.top_idx, self.top_logprob, self.status)
        self._device = _device_of(self.entropy)
        self._stream = _stream_of(self._device)

    def __call__(self, z: torch.Tensor, tokens: torch.Tensor | None = None):
        """(logprob [n, n_tokens], entropy [n], top_idx [n, top_k], top_logprob [n, top_k])."""
        n, s, dev = _rows("z", z, self.N), self.n_tokens, self._device
        ld = _matrix("z", z, self.dtype, dev, n, self.V)
        t = None
        if s > 0:
            if tokens is None:
                raise ValueError("tokens must be given for n_tokens > 0")
            t = _list("tokens", tokens, torch.int32, dev, n, s)
        code = self._lib.tw_token_logprobs(
            z.data_ptr(), ld, n, self.V, self._dt, t, s, self.temperature, self.top_k, *self._to, self._stream())
        if code:
            _lib.check(code, "tw_token_logprobs")
        if n == self.N:
            return self.logprob, self.entropy, self.top_idx, self.top_logprob
        return self.logprob[:n], self.entropy[:n], self.top_idx[:n], self.top_logprob[:n]


def token_logprobs(z, tokens=None, top_k: int = 0, temperature: float = 1.0):
    """One-shot form; tokens [n] or [n, s]. Returns (logprob, entropy, top_idx, top_logprob, status)."""
    n = z.shape[0]
    if tokens is None:
        s = 0
    elif tokens.dim() == 2 and tokens.shape[0] == n:
        s = tokens.shape[1]
    else:  # at least one, so that tokens for fewer rows are refused
        s = max(1, tokens.numel() // max(n, 1))
    op = TokenLogprobs(n, z.shape[1], s, top_k, temperature, z.dtype, z.device)
    return (*op(z, tokens), op.status)
