"""Inference forwards of other list lengths from several host threads at once, through the C
entry point: each launch's shared memory is its own."""
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402
from test_gpu_row_ops_threads import _at_once  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _forward(C, gated, keep):
    T, d, I, W = 8, 256, 4096, 128
    f = tw.TwellFFN(T, d, I, W, C)
    x = torch.randn(T, d, device="cuda").bfloat16()
    Wg, Wu, Wd = (torch.randn(I, d, device="cuda").mul_(0.05).bfloat16() for _ in range(3))
    keep += [f, x, Wg, Wu, Wd]
    want = f(x, Wg, Wu if gated else None, Wd).clone()
    call = tw.load().twell_ffn_fwd, (x.data_ptr(), Wg.data_ptr(), Wu.data_ptr() if gated else None, Wd.data_ptr(), T, d, I,
                                     W, C, f.ovf_cap, f._tws, f.ws.data_ptr(), f.ws_bytes, f.y.data_ptr(),
                                     f.status.data_ptr())
    return call, f, want


@pytest.mark.parametrize("gated", [True, False])
def test_threads_with_other_list_lengths(gated):
    keep = []
    made = [_forward(C, gated, keep) for C in (128, 96) * 3]
    assert _at_once([m[0] for m in made], 2000) == {_lib.TW_OK}
    for _, f, want in made:
        tw.raise_if_device_error(f.status)
        assert torch.equal(f.y, want)
