"""What an embedding gradient is added to was written by someone: by the caller, or zeros."""
import os

import pytest

import activation_sparse_feedforward_gb300 as tw

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()


def test_an_objects_gradient_is_zero_before_the_first_call():
    was = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # torch.empty is then filled with NaN
    try:
        op = tw.Embedding(4, 6, 8, device="cpu")
    finally:
        torch.use_deterministic_algorithms(was)
    assert not op.dweight.any()


def test_one_shot_add_without_a_gradient_is_refused():
    with pytest.raises(ValueError, match="add needs `out`"):
        tw.embedding_bwd(torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), 6, add=True)
