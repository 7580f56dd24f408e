"""Calls of other sizes from several host threads at once, through the C entry points: each
launch's shared memory is its own, whatever another thread asks of the same kernel."""
import threading

import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _at_once(calls, times):
    """Each call (function, arguments without the stream) `times` times on a thread and a
    stream of its own; the status codes that came back."""
    codes, start = set(), threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(call, stream):
        function, args = call
        args = (*args, stream.cuda_stream)
        start.wait()
        for _ in range(times):
            codes.add(function(*args))

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return codes


def _distill(N, V, keep):
    z, dz = torch.randn(N, V, device="cuda"), torch.empty(N, V, device="cuda")
    labels, loss = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.empty(N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep += [z, dz, labels, loss, status]
    return tw.load().tw_distill, (z.data_ptr(), V, N, V, _lib.TW_F32, None, None, 0, 0, None, labels.data_ptr(), 1.0, 0.0,
                                  1.0, None, 1.0, loss.data_ptr(), dz.data_ptr(), V, status.data_ptr())


def _norm_fwd(T, d, residual, keep):
    x, r, y = (torch.randn(T, d, device="cuda") for _ in range(3))
    keep += [x, r, y]
    return tw.load().tw_layer_norm_fwd, (x.data_ptr(), d, r.data_ptr() if residual else None, d, None, None, T, d, 1e-5,
                                         _lib.TW_F32, _lib.TW_F32, None, 0, y.data_ptr(), d, None, None)


def _norm_bwd(T, d, residual, keep):
    x, dy, r, dx = (torch.randn(T, d, device="cuda") for _ in range(4))
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    keep += [x, dy, r, dx, mean, rstd]
    return tw.load().tw_layer_norm_bwd, (dy.data_ptr(), d, x.data_ptr(), d, mean.data_ptr(), rstd.data_ptr(), None,
                                         r.data_ptr() if residual else None, d, T, d, _lib.TW_F32, _lib.TW_F32,
                                         dx.data_ptr(), d, None, None, None, 0)


# pairs that share a kernel and want other amounts of shared memory of it, both above what
# any kernel may have without asking
@pytest.mark.parametrize("pair", ["distill", "norm_fwd", "norm_bwd"])
def test_threads_with_other_sizes(pair):
    keep = []
    calls = dict(distill=lambda: [_distill(4, 140000, keep), _distill(4, 100000, keep)],
                 norm_fwd=lambda: [_norm_fwd(16, 2048, True, keep), _norm_fwd(16, 2048, False, keep)],
                 norm_bwd=lambda: [_norm_bwd(400, 2048, True, keep), _norm_bwd(400, 2048, False, keep)])[pair]()
    assert _at_once(calls * 3, 4000) == {_lib.TW_OK}
