"""An Orthogonalize object called with fewer matrices than it was made for: another layout of the
same workspace (units, slices, counters), whatever the calls before have left there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import updates  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(64, 64), (300, 520), (704, 256), (1100, 900)])
def test_any_number_up_to_the_objects(m, n):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    rng = np.random.default_rng(m + n)
    draw = lambda: torch.from_numpy(rng.normal(size=(m, n)).astype(np.float32)).cuda()  # noqa: E731
    gs, bufs = [draw() for _ in range(8)], [draw() for _ in range(8)]
    op = tw.Orthogonalize(m, n, count=8, dtype=torch.float32)
    guarded = torch.full((op.ws_bytes + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    op.ws = guarded[:op.ws_bytes]
    op._to = op._to[0], op.ws.data_ptr(), op._to[2]
    for k, fill in ((1, 255), (8, 255), (2, None), (1, None), (5, 0), (3, None), (8, None), (1, None)):
        if fill is not None:
            op.ws.fill_(fill)
        ours, theirs = [b.clone() for b in bufs[:k]], [b.clone() for b in bufs[:k]]
        outs = [o.clone() for o in op(gs[:k], ours)]
        want = tw.Orthogonalize(m, n, count=k, dtype=torch.float32)(gs[:k], theirs)
        assert len(outs) == k
        for i in range(k):
            assert torch.equal(outs[i], want[i]) and torch.equal(ours[i], theirs[i])
        # the last of them against the definition (each product's three roundings, test_gpu_ortho.py)
        u = gs[k - 1].double() + 0.95 * ours[-1].double()
        ref = updates.newton_schulz(u.cpu().numpy())
        err = np.linalg.norm(outs[-1].double().cpu().numpy() - ref) / np.linalg.norm(ref)
        assert err <= 15 * 2.0 ** -12, (k, err)
        assert (guarded[op.ws_bytes:] == 0x5A).all()
    assert op.status.item() == 0
