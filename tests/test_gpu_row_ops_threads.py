"""Calls of other sizes from two host threads at once: each launch's shared memory is its own."""
import threading

import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _at_once(calls, times):
    """Runs each call `times` times on a thread and a stream of its own; what they raised."""
    raised, start = [], threading.Barrier(len(calls))
    torch.cuda.synchronize()

    def work(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for n in range(times):
                    call()
                    if n % 64 == 63:
                        torch.cuda.current_stream().synchronize()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the test)
            raised.append(repr(e))

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def _distill(N, V, K):
    z = torch.randn(N, V, device="cuda")
    labels = torch.zeros(N, dtype=torch.int32, device="cuda")
    op = tw.DistillLoss(N, V, 0, dtype=torch.float32, kd_weight=0.0, ce_weight=1.0)
    return lambda: op.forward_backward(z, labels=labels)


def _norm(T, d, residual, backward):
    x = torch.randn(T, d, device="cuda")
    r = torch.randn(T, d, device="cuda") if residual else None
    op = tw.LayerNorm(T, d, dtype=torch.float32)
    if not backward:
        return lambda: op.forward(x, residual=r)
    op.forward(x)
    return lambda: op.backward(x, x, dres=r)


# pairs of one kernel with other sizes of shared memory, both above what needs no leave
@pytest.mark.parametrize("pair", ["distill_cluster", "distill_rows", "norm_fwd", "norm_bwd"])
def test_two_threads_with_other_sizes(pair):
    calls = dict(distill_cluster=lambda: (_distill(8, 140000, 0), _distill(8, 100000, 0)),
                 distill_rows=lambda: (_distill(320, 1000, 0), _distill(320, 12000, 0)),
                 norm_fwd=lambda: (_norm(64, 2048, True, False), _norm(64, 2048, False, False)),
                 norm_bwd=lambda: (_norm(400, 2048, True, True), _norm(400, 2048, False, True)))[pair]()
    assert _at_once(calls, 3000) == []
