"""Torch-facing binding of the operators on weight matrices: orthogonalised updates (see
tw_orthogonalize in include/twell.h).

As in ``ops``: objects preallocate every buffer, calls enqueue on torch's current stream
and neither allocate nor synchronise. Every operand is on the object's device, and that is
the current one; else ValueError. An object's workspace serves one call at a time: calls on
two streams, or two captured graphs replayed at once, need an object each.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .ops import _workspace
from .row_ops import _device_of, _dtype_code, _matrix, _stream_of

#: the quintic step that K. Jordan published in 2024 for orthogonalised momentum (five of them):
#: singular values in (0, 1] end in about [0.7, 1.2]
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


class Orthogonalize:
    """Preallocated orthogonalised update of up to `count` matrices [m, n] at once, as
    optimisers of hidden weights take them (momentum, then Newton-Schulz steps; see
    tw_orthogonalize).

    dtype: the type of the result. grad_dtype: of the gradients (the layer's are float32).
    momentum, nesterov: how a call with buffers mixes them in. coefficients: one (a, b, c)
    for all steps, or one for each; tw_orthogonalize says how precise the result is. `status`
    gets TW_ETIMEOUT if a bounded wait ran out.
    """

    def __init__(self, m: int, n: int, count: int = 1, dtype: torch.dtype = torch.bfloat16,
                 grad_dtype: torch.dtype = torch.float32, steps: int = 5, coefficients=COEFFICIENTS,
                 momentum: float = 0.95, nesterov: bool = True, device="cuda"):
        self.m, self.n, self.count, self.dtype, self.grad_dtype = m, n, count, dtype, grad_dtype
        self.steps, self.momentum, self.nesterov = int(steps), float(momentum), bool(nesterov)
        self._dt, self._gdt = _dtype_code(dtype), _dtype_code(grad_dtype)
        if m < 1 or n < 1 or not 1 <= count <= _lib.TW_ORTHO_MOST:
            raise ValueError(f"m and n must be positive and count 1 to {_lib.TW_ORTHO_MOST}, got {(m, n, count)}")
        if not 1 <= self.steps <= 32:
            raise ValueError(f"steps must be 1 to 32, got {steps}")
        rows = list(coefficients)
        if not any(hasattr(r, "__len__") for r in rows):
            rows = [rows] * self.steps
        if len(rows) != self.steps or any(not hasattr(r, "__len__") or len(r) != 3 for r in rows):
            raise ValueError("coefficients must be three numbers, or three for each step")
        self.coefficients = [tuple(float(v) for v in r) for r in rows]
        self._coef = (ctypes.c_float * (3 * self.steps))(*[v for r in self.coefficients for v in r])
        self._lib = _lib.load()
        self.ws_bytes = int(self._lib.tw_orthogonalize_workspace_size(m, n, count))
        if self.ws_bytes == 0:
            raise ValueError(f"unsupported size {(m, n)}: at most 16384 by 2^20")
        self.out = [torch.empty((m, n), dtype=dtype, device=device) for _ in range(count)]
        self.ws = _workspace(self.ws_bytes, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._addresses = ctypes.c_void_p * count
        self._to = [t.data_ptr() for t in self.out], self.ws.data_ptr(), self.status.data_ptr()
        self._device = _device_of(self.status)
        self._stream = _stream_of(self._device)

    def _list(self, name, tensors, dtype, k):
        """The addresses of k matrices and their common row stride."""
        if len(tensors) != k:
            raise ValueError(f"{name} has {len(tensors)} matrices, expected {k}")
        strides = [_matrix(f"{name}[{i}]", t, dtype, self._device, self.m, self.n) for i, t in enumerate(tensors)]
        if any(ld != strides[0] for ld in strides):
            raise ValueError(f"{name} must have one row stride, got {strides}")
        if strides[0] < self.n:
            raise ValueError(f"{name} must not have overlapping rows")
        return [t.data_ptr() for t in tensors], strides[0]

    def __call__(self, grads, buffers=None, out=None, scale: float = 1.0, beta: float = 0.0):
        """The updates of `grads`, a list of matrices (or one, and one is returned): new
        momentum into `buffers` (float32, in place; None: no momentum), results into `out`
        (beta out + scale X; None: the object's own, beta 0)."""
        single = isinstance(grads, torch.Tensor)
        if single:
            grads, buffers, out = [grads], None if buffers is None else [buffers], None if out is None else [out]
        k = len(grads)
        if not 1 <= k <= self.count:
            raise ValueError(f"expected 1 to {self.count} matrices, got {k}")
        if buffers is None and self.momentum != 0.0:
            raise ValueError("buffers must be given, or momentum 0")
        if out is None and beta != 0.0:
            raise ValueError("beta needs `out`")
        arr = self._addresses
        g, ldg = self._list("grads", grads, self.grad_dtype, k)
        b, ldb = (None, 0) if buffers is None else self._list("buffers", buffers, torch.float32, k)
        to, ws, status = self._to
        o, ldo = (to, self.n) if out is None else self._list("out", out, self.dtype, k)
        code = self._lib.tw_orthogonalize(
            arr(*g), ldg, self._gdt, None if b is None else arr(*b), ldb, self.momentum, self.nesterov, k, self.m, self.n,
            self.steps, self._coef, scale, beta, arr(*o[:k]), ldo, self._dt, ws, self.ws_bytes, status, self._stream())
        if code:
            _lib.check(code, "tw_orthogonalize")
        out = self.out[:k] if out is None else out
        return out[0] if single else list(out)


def orthogonalize(grad, buffer=None, dtype: torch.dtype = torch.bfloat16, steps: int = 5, coefficients=COEFFICIENTS,
                  momentum: float = 0.95, nesterov: bool = True, scale: float = 1.0):
    """One-shot form for one matrix (buffer None: without momentum). Returns (update, status)."""
    op = Orthogonalize(grad.shape[0], grad.shape[1], 1, dtype, grad.dtype, steps, coefficients,
                       momentum if buffer is not None else 0.0, nesterov, device=grad.device)
    return op(grad, buffer, scale=scale), op.status
