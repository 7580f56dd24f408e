"""The binding refuses lists that lie the wrong way round: n rows of k entries are wanted, and a
[k, n] array holds as many elements."""
import pytest

torch = pytest.importorskip("torch")

from test_row_ops_devices import CALLS, Notes, OnGpu, _operands, current_device  # noqa: E402, F401


@pytest.mark.parametrize("which,operand", [("distill", "idx"), ("distill", "val"), ("logprobs", "tokens")])
def test_lists_the_wrong_way_round_are_refused(which, operand, current_device):  # noqa: F811
    notes = Notes()
    a = _operands(which, 0)
    (rows, entries), dtype = CALLS[which][2][operand]
    a[operand] = OnGpu(torch.zeros((entries, rows), dtype=dtype), 0)
    with pytest.raises(ValueError, match="expected"):
        CALLS[which][1](CALLS[which][0](notes, 0), a)
    assert not notes.calls
    a[operand] = OnGpu(torch.zeros(rows * entries, dtype=dtype), 0)  # in one dimension, as they lie in memory
    CALLS[which][1](CALLS[which][0](notes, 0), a)
    assert len(notes.calls) == 1
