"""A part of the distillation whose weight is 0 is not looked at: its operands may be absent."""
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from test_row_ops_devices import Notes, OnGpu, current_device  # noqa: E402, F401

N, V, K = 4, 8, 3


def _op(kd, ce):
    op = tw.DistillLoss(N, V, K, kd_weight=kd, ce_weight=ce, device="cpu")
    op._lib, op._device, op._stream = Notes(), 0, lambda: 0
    return op


def test_no_list_is_asked_for_without_the_teachers_part(current_device):  # noqa: F811
    z, labels = OnGpu(torch.zeros(N, V).bfloat16(), 0), OnGpu(torch.zeros(N, dtype=torch.int32), 0)
    op = _op(0.0, 1.0)
    op.forward_backward(z, labels=labels)
    assert op._lib.calls == ["tw_distill"]


def test_a_list_is_asked_for_with_it(current_device):  # noqa: F811
    op = _op(0.5, 0.5)
    with pytest.raises(ValueError, match="idx and val"):
        op.forward_backward(OnGpu(torch.zeros(N, V).bfloat16(), 0))
    assert not op._lib.calls


def test_the_list_is_passed_on_with_it(current_device):  # noqa: F811
    z = OnGpu(torch.zeros(N, V).bfloat16(), 0)
    idx, val = OnGpu(torch.zeros(N, K, dtype=torch.int32), 0), OnGpu(torch.zeros(N, K), 0)
    op = _op(0.5, 0.0)
    op.forward_backward(z, idx, val)
    assert op._lib.calls == ["tw_distill"]
