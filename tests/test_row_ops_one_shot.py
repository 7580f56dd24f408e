"""The one-shot log probabilities take n tokens a row from the tokens' shape: tokens for fewer
rows than the logits have are refused, not left out."""
import pytest

import activation_sparse_feedforward_gb300 as tw
from activation_sparse_feedforward_gb300 import row_ops

torch = pytest.importorskip("torch")


@pytest.fixture
def taken(monkeypatch):
    """(n_tokens, tokens) of each call, in place of the call."""
    seen = []

    class Op:
        status = None

        def __init__(self, N, V, n_tokens, *a):
            self.n_tokens = n_tokens

        def __call__(self, z, tokens):
            seen.append((self.n_tokens, tokens))
            if self.n_tokens > 0 and tokens.numel() != z.shape[0] * self.n_tokens:  # as the operator does
                raise ValueError("tokens")
            return ()

    monkeypatch.setattr(row_ops, "TokenLogprobs", Op)
    return seen


@pytest.mark.parametrize("rows,shape,each", [(4, (4,), 1), (4, (4, 3), 3), (4, (4, 0), 0), (1, (5,), 5), (0, (0, 3), 3),
                                             (0, (0,), 1), (2, (2, 1), 1)])
def test_tokens_a_row(rows, shape, each, taken):
    tw.token_logprobs(torch.zeros(rows, 8), torch.zeros(shape, dtype=torch.int32))
    assert taken[0][0] == each


@pytest.mark.parametrize("shape", [(2,), (3,), (1, 2), (0,), (5,), (3, 1)])
def test_tokens_for_other_rows_are_refused(shape, taken):
    with pytest.raises(ValueError):
        tw.token_logprobs(torch.zeros(4, 8), torch.zeros(shape, dtype=torch.int32))


def test_no_tokens(taken):
    tw.token_logprobs(torch.zeros(4, 8))
    assert taken == [(0, None)]
