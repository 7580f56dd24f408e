"""A wait of the orthogonalised update that runs out on the GPU, and what comes after it.

tw_orthogonalize_timeout_probe has the first square wait for a block that no one writes. Every
CTA gives up within the library's limit (1 s) and returns: TW_ETIMEOUT in the status word, the
result untouched. The next call on the same workspace and stream gives the usual bits."""
import os
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402

P = 4096  # fake, aligned, never dereferenced


def test_refusals():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()
    lib = tw.load()
    need = lib.tw_orthogonalize_workspace_size(64, 64, 1)
    good = dict(grad=P, m=64, n=64, out=P, ws=P, ws_bytes=need, status=P)
    for kw, code in ((dict(m=0), "EINVAL"), (dict(m=(1 << 20) + 1), "EUNSUPPORTED"), (dict(grad=None), "EINVAL"), (dict(out=P + 2), "EALIGN"),
                     (dict(ws=None), "EINVAL"), (dict(ws_bytes=10), "EWORKSPACE"), (dict(status=None), "EINVAL")):
        assert lib.tw_orthogonalize_timeout_probe(*{**good, **kw}.values(), None) == getattr(_lib, "TW_" + code), kw


# one 256-wide tile in slices; several tiles, of a wide matrix; more tiles than pairs of SMs
@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(300, 200), (700, 1300), (6000, 2100)])
def test_a_withheld_block_times_out_and_the_workspace_recovers(m, n):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    lib = tw.load()
    g = torch.from_numpy(np.random.default_rng(m).normal(size=(m, n)).astype(np.float32)).cuda()
    op = tw.Orthogonalize(m, n, momentum=0.0, dtype=torch.float32)
    want = op(g).clone()
    out = torch.full((m, n), 7.0, device="cuda")
    torch.cuda.synchronize()
    t0 = time.monotonic()
    code = lib.tw_orthogonalize_timeout_probe(g.data_ptr(), m, n, out.data_ptr(), op.ws.data_ptr(), op.ws_bytes, op.status.data_ptr(),
                                              torch.cuda.current_stream().cuda_stream)
    assert code == _lib.TW_OK
    torch.cuda.synchronize()
    elapsed = time.monotonic() - t0
    assert op.status.item() == _lib.TW_ETIMEOUT
    assert 0.5 < elapsed < 30.0, elapsed
    assert (out == 7.0).all()
    op.status.zero_()
    for _ in range(2):
        assert torch.equal(op(g), want)
    assert op.status.item() == 0
