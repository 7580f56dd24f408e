"""The binding refuses operands that are not where the object's buffers are, and a current
device that is another, before anything reaches the library. The operands here are stand-ins
that say they are on a GPU; the library is one that notes its calls."""
import pytest

import activation_sparse_feedforward_gb300 as tw
from activation_sparse_feedforward_gb300 import row_ops

torch = pytest.importorskip("torch")

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
N, V, K, S = 4, 8, 3, 2


class OnGpu:
    """A host tensor that says it is on a GPU."""

    def __init__(self, t, index):
        self._t, self._index = t, index
        self.dtype, self.shape, self.is_cuda = t.dtype, t.shape, True

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        return getattr(self._t, name)


class Notes:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def current_device(monkeypatch):
    at = [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return at


def _norm(notes, index):
    op = tw.LayerNorm(N, V, device="cpu")
    op._lib, op._device, op._stream = notes, index, row_ops._stream_of(index)
    return op


def _distill(notes, index):
    op = tw.DistillLoss(N, V, K, ce_weight=1.0, device="cpu")
    op._lib, op._device, op._stream = notes, index, row_ops._stream_of(index)
    return op


def _logprobs(notes, index):
    op = tw.TokenLogprobs(N, V, n_tokens=S, top_k=2, device="cpu")
    op._lib, op._device, op._stream = notes, index, row_ops._stream_of(index)
    return op


MATRIX, VECTOR = ((N, V), BF16), ((N,), F32)
CALLS = {
    "norm_fwd": (_norm, lambda op, a: op.forward(a["x"], a["weight"], a["bias"], residual=a["residual"]),
                 dict(x=MATRIX, weight=((V,), BF16), bias=((V,), BF16), residual=MATRIX)),
    "norm_bwd": (_norm, lambda op, a: op.backward(a["dy"], a["x"], a["weight"], a["dres"], a["mean"], a["rstd"]),
                 dict(dy=MATRIX, x=MATRIX, weight=((V,), BF16), dres=MATRIX, mean=VECTOR, rstd=VECTOR)),
    "distill": (_distill, lambda op, a: op.forward_backward(a["z"], a["idx"], a["val"], a["rest"], a["labels"], a["dloss"],
                                                            out=a["out"]),
                dict(z=MATRIX, idx=((N, K), I32), val=((N, K), F32), rest=VECTOR, labels=((N,), I32), dloss=VECTOR, out=MATRIX)),
    "logprobs": (_logprobs, lambda op, a: op(a["z"], a["tokens"]), dict(z=MATRIX, tokens=((N, S), I32))),
}


def _operands(which, index, **other):
    shapes = CALLS[which][2]
    return {k: OnGpu(torch.zeros(shape, dtype=dtype), other.get(k, index)) for k, (shape, dtype) in shapes.items()}


@pytest.mark.parametrize("which", CALLS)
def test_operands_on_the_objects_device_reach_the_library(which, current_device):
    for index in (0, 1):
        current_device[0] = index
        notes = Notes()
        CALLS[which][1](CALLS[which][0](notes, index), _operands(which, index))
        assert len(notes.calls) == 1


@pytest.mark.parametrize("which,operand", [(w, o) for w in CALLS for o in CALLS[w][2]])
def test_an_operand_on_another_device_is_refused(which, operand, current_device):
    notes = Notes()
    with pytest.raises(ValueError, match=f"{operand} must be .*device"):
        CALLS[which][1](CALLS[which][0](notes, 0), _operands(which, 0, **{operand: 1}))
    assert not notes.calls


@pytest.mark.parametrize("which", CALLS)
def test_an_object_with_host_buffers_is_refused(which, current_device):
    notes = Notes()
    op = CALLS[which][0](notes, 0)
    op._device = row_ops._device_of(torch.empty(1))
    for index in (0, -1):  # the operands on a GPU, and on the host too
        with pytest.raises(ValueError, match="CUDA"):
            CALLS[which][1](op, _operands(which, index))
    assert not notes.calls


@pytest.mark.parametrize("which", CALLS)
def test_another_current_device_is_refused(which, current_device):
    current_device[0] = 1
    notes = Notes()
    with pytest.raises(ValueError, match="current device"):
        CALLS[which][1](CALLS[which][0](notes, 0), _operands(which, 0))
    assert not notes.calls


def test_objects_know_their_device():
    for op in (tw.LayerNorm(N, V, device="cpu"), tw.DistillLoss(N, V, K, device="cpu"), tw.TokenLogprobs(N, V, device="cpu")):
        assert op._device not in (0, 1, torch.empty(1).get_device())
