"""The workspace of RMS norm's backward holds the widest form's partial sums: a row off 16 bytes
takes the threads of up to E - 1 columns more than it has (E elements in 16 bytes), so that its
team may be the next wider one."""
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import ends  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
#: the columns that a team holds, 16 (or 8) a thread
TEAMS = [512, 1024, 1536, 2048, 2560, 4096, 5120, 5632, 7168, 8192]


def test_a_partial_is_as_wide_as_the_team():
    if not os.path.exists(tw.lib_path()):
        from activation_sparse_feedforward_gb300.build import build
        build()
    lib = tw.load()
    for d in range(1, 8185):
        team = next(t for t in TEAMS if d + 7 <= t)
        assert lib.tw_rms_norm_bwd_workspace_size(512, d) >= 4 * 512 * team, d
    for d in (1, 64, 1018, 1024, 4090, 8192, 9001, 16384):
        sizes = [lib.tw_rms_norm_bwd_workspace_size(T, d) for T in (1, 2, 77, 511, 512, 513, 1 << 30)]
        assert sizes == sorted(sizes) and sizes[-1] == sizes[-3]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [505, 509, 512, 1017, 1018, 1021, 1023, 1024, 1530, 2042, 2047, 2048, 2557, 4090, 4096, 5117, 8184])
def test_nothing_behind_the_workspace_is_written(d, dtype):
    """Rows one element off 16 bytes in every matrix; guards behind the workspace."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    T, guard = 700, 1 << 20
    rng = np.random.default_rng(d)

    def off(fill=None):
        t = torch.empty(T * d + 1, dtype=dtype, device="cuda")
        if fill is not None:
            t[1:] = torch.from_numpy(fill.astype(np.float32)).to(dtype).cuda().view(-1)
        return t[1:].view(T, d)

    x, dy = off(rng.normal(size=(T, d))), off(rng.normal(size=(T, d)))
    lib = tw.load()
    need = lib.tw_rms_norm_bwd_workspace_size(T, d)
    ws = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dw = off(), torch.empty(d, device="cuda")
    code = {BF16: 1, F32: 0}[dtype]
    st = lib.tw_rms_norm_bwd(dy.data_ptr(), d, x.data_ptr(), d, rstd.data_ptr(), None, None, 0, T, d, code, code, dx.data_ptr(), d,
                             dw.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert (ws[need:] == 0x5A).all()
    want_dx, want_dw = ends.rms_norm_grad(dy.double().cpu().numpy(), x.double().cpu().numpy())
    # a sum of T products, each of two roundings, and dx rounded to its type: a norm of the whole
    # (sums of d for the one number that dx shares along a row)
    u = 2.0 ** -8 if dtype is BF16 else 2.0 ** -24
    for got, want, tol in ((dx, want_dx, u + d * 2.0 ** -24), (dw, want_dw, (T + 4) * 2.0 ** -24)):
        err = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert err <= tol, err
