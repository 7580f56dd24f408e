"""The weight's and bias's gradients are sums over rows in a fixed order for each form of a
call: rows on 16 bytes and off it, dx of its own and in place of dy. Each form repeats its bits;
the forms agree within the bound of two fp32 sums of T products in any order: (2 T + 8) 2^-24 of
the sum of magnitudes (a product and its two factors are rounded to 2^-24 each)."""
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _off16(t):
    """The same rows, one element past 16 bytes."""
    buf = torch.zeros((t.shape[0], t.shape[1] + 8), dtype=t.dtype, device="cuda")
    buf[:, 1:1 + t.shape[1]] = t
    return buf[:, 1:1 + t.shape[1]]


# rows of the one-launch kernel in both forms, in the aligned one alone, and in neither
@pytest.mark.parametrize("T,d", [(77, 512), (250, 1024), (400, 2048), (3000, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_form_repeats_its_bits(T, d, dtype):
    g = torch.Generator("cuda").manual_seed(T)
    x, dy, dres = (torch.randn(T, d, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = torch.randn(d, device="cuda", generator=g)
    ln = tw.LayerNorm(T, d, dtype=dtype, weight_dtype=torch.float32)
    ln.forward(x, w)
    lib, stream = tw.load(), torch.cuda.current_stream().cuda_stream
    code = {torch.bfloat16: 1, torch.float32: 0}[dtype]

    def run(x, dy, in_place):
        dy = dy.clone() if dy.is_contiguous() else _off16(dy)
        dx = dy if in_place else torch.empty_like(x)
        dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        r = lib.tw_layer_norm_bwd(dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), ln.mean.data_ptr(),
                                  ln.rstd.data_ptr(), w.data_ptr(), dres.data_ptr(), d, T, d, code, 0, dx.data_ptr(),
                                  dx.stride(0), dw.data_ptr(), db.data_ptr(), ln.ws.data_ptr(), ln.ws_bytes, stream)
        assert r == 0
        return dw, db

    xh = (x.double() - ln.mean.double()[:, None]) * ln.rstd.double()[:, None]
    size_w, size_b = (dy.double() * xh).abs().sum(0), dy.double().abs().sum(0)
    bound = (2 * T + 8) * 2.0 ** -24
    first = None
    for xs, dys in ((x, dy), (_off16(x), _off16(dy))):
        for in_place in (False, True):
            want = run(xs, dys, in_place)
            for _ in range(5):
                again = run(xs, dys, in_place)
                assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
            first = first or want
            assert ((want[0] - first[0]).double().abs() <= bound * size_w).all()
            assert ((want[1] - first[1]).double().abs() <= bound * size_b).all()
