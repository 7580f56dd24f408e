"""Calls of other sizes from several host threads at once, each on its own stream and object:
embedding gradients (whose sort's shared memory goes by the vocabulary), RMS norms (whose ring
goes by the width) and orthogonalised updates give what they give alone."""
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


def _calls():
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    calls = []
    for T, V, d in ((700, 5000, 64), (3000, 150000, 32), (900, 64, 100)):
        op, dy = tw.Embedding(T, V, d), rand(T, d).bfloat16()
        tok = torch.randint(-1, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
        calls.append(lambda op=op, dy=dy, tok=tok: op.backward(dy, tok))
    for T, d, kw in ((300, 8192, {}), (300, 512, {}), (300, 8192, dict(fp8=True, group=128, backward=False))):
        op, x = tw.RMSNorm(T, d, **kw), rand(T, d).bfloat16()
        f = op.forward_fp8 if kw else op.forward
        calls.append(lambda f=f, x=x: f(x)[0].view(torch.uint8))
    for m, n in ((300, 200), (1000, 1200)):
        op, g = tw.Orthogonalize(m, n, momentum=0.0), rand(m, n)
        calls.append(lambda op=op, g=g: op(g))
    return calls


def test_each_gives_what_it_gives_alone():
    calls = _calls()
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    streams, start = [torch.cuda.Stream() for _ in calls], threading.Barrier(len(calls))
    wrong = []

    def work(i):
        start.wait()
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got = calls[i]().clone()
            streams[i].synchronize()
        if not torch.equal(got, want[i]):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
