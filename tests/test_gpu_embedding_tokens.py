"""Tokens of any int32 value, and one object for batches of many lengths."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402
from oracle import ends  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


@pytest.mark.parametrize("T", [300, 3000])
@pytest.mark.parametrize("V", [1, 77, 5003, 160000])
@pytest.mark.parametrize("add", [False, True])
def test_the_ends_of_the_type_are_outside(T, V, add):
    rng = np.random.default_rng(V)
    tok = rng.integers(0, V, T)
    bad = np.array([-2 ** 31, -2 ** 31 + 1, -2 ** 31 + V, -V, -2, V, 2 * V, 2 ** 31 - V, 2 ** 31 - 1])
    where = rng.random(T) < 0.5
    given = np.where(where, rng.choice(bad[(bad < -1) | (bad >= V)], T), tok).astype(np.int32)
    none = torch.from_numpy(np.where(where, -1, tok).astype(np.int32)).cuda()
    dy, w = torch.randn(T, 40, device="cuda"), torch.randn(V, 40, device="cuda")
    op = tw.Embedding(T, V, 40, dtype=F32)
    old = torch.randn(V, 40, device="cuda")
    y, dw = op.forward(none, w).clone(), op.backward(dy, none, out=old.clone(), add=add)
    assert op.status.item() == 0
    given = torch.from_numpy(given).cuda()
    for call, want in ((lambda: op.forward(given, w), y), (lambda: op.backward(dy, given, out=old.clone(), add=add), dw)):
        assert torch.equal(call(), want)
        assert op.status.item() == _lib.TW_EINVAL
        op.status.zero_()


@pytest.mark.parametrize("d,dtype", [(64, BF16), (1027, BF16), (2048, F32)])
@pytest.mark.parametrize("add", [False, True])
def test_one_object_for_batches_of_many_lengths(d, dtype, add):
    """Shorter batches go in other chunks of the same workspace, whatever it holds."""
    rng = np.random.default_rng(d)
    V, most = 1009, 9700
    op = tw.Embedding(most, V, d, dtype=dtype, scale=0.5)
    guarded = torch.full((op.ws_bytes + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    op.ws = guarded[:op.ws_bytes]
    op._to_bwd = (op._to_bwd[0], op.ws.data_ptr())
    dy = torch.from_numpy(rng.normal(size=(most, d)).astype(np.float32)).to(dtype).cuda()
    tok = np.minimum(np.exp(rng.random(most) * np.log(V + 1)).astype(np.int64) - 1, V - 1)
    tok[rng.random(most) < 0.05] = -1
    for T in (9700, 4800, 513, 77, 9600, 2001, 1, 9700):
        op.ws.fill_(0xFF)
        old = torch.from_numpy(rng.normal(size=(V, d)).astype(np.float32)).cuda()
        tokens = torch.from_numpy(tok[:T].astype(np.int32)).cuda()
        got = op.backward(dy[:T], tokens, out=old.clone(), add=add).double().cpu().numpy()
        f64 = dy[:T].double().cpu().numpy()
        ref, mag = ends.embedding_grad(f64, tok[:T], V, 0.5), ends.embedding_grad(np.abs(f64), tok[:T], V, 0.5)
        # n rows added one after the other, the scale, and what was there: a rounding each
        n = np.bincount(tok[:T][tok[:T] >= 0], minlength=V)[:, None]
        tol = (n + 2) * 2.0 ** -24 * mag
        if add:
            was = old.double().cpu().numpy()
            ref, tol = ref + was, tol + 2.0 ** -24 * (np.abs(was) + mag)
        assert (np.abs(got - ref) <= tol).all(), T
        assert (guarded[op.ws_bytes:] == 0x5A).all()
    assert op.status.item() == 0
