"""GPU parity of the distillation loss and of token log probabilities against
oracle/ends.py in float64.

Tolerances, from the arithmetic. A row's exponentials e = 2^(c z - M) carry, relative,
the hardware exponential (2^-22), the fused exponent's rounding and c's own (2^-24 of an
exponent below 2^7: 2^-16 at the far tail, 2^-24 near the maximum, weighted by e) and
the sums' roundings, at most about 200 sequential positive terms a thread and the trees:
together below R = 400 * 2^-24 of a probability. A logarithm of them is off by R plus
2^-22 of the exponents' size. u is the unit roundoff of the type that dz is rounded to.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from activation_sparse_feedforward_gb300 import _lib  # noqa: E402
from oracle import ends  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 1e-38, F16: 2.0 ** -25, F32: 1e-38}
R = 400 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw.load()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _logits(rng, N, V, dtype, pad=0, off=0, scale=2.5):
    full = torch.from_numpy(rng.normal(0, scale, (N, V + pad + off)).astype(np.float32)).to(dtype).cuda()
    return full[:, off:off + V]


def _teacher(rng, z, K, ragged=True):
    N, V = z.shape
    t = _f64(z) + rng.normal(0, 1, (N, V))
    idx = np.argsort(-t, axis=1)[:, :K].astype(np.int32)
    val = np.take_along_axis(t, idx, 1).astype(np.float32)
    if ragged and N > 2 and K > 1:
        idx[1, K // 2:] = -1
        idx[2, :] = -1
    return torch.from_numpy(idx).cuda(), torch.from_numpy(val).cuda()


def _log_tol(z, tau):
    zf = _f64(z)
    zf = np.where(np.isfinite(zf), zf, 0)
    return R + 2.0 ** -22 * (np.abs(zf).max() / min(tau, 1.0) * 1.4427 + 20)


def _check_distill(loss, dz, z, idx, val, rest, labels, tau, kd, ce, dloss=None, scale=1.0):
    n = lambda t: None if t is None else _f64(t)  # noqa: E731
    i = None if idx is None else idx.cpu().numpy()
    lab = None if labels is None else labels.cpu().numpy()
    Z = _f64(z)
    rl, rd = ends.distill(Z, i, n(val), n(rest), lab, tau, kd, ce, n(dloss), scale)
    if loss is not None:
        got = _f64(loss)
        fin = np.isfinite(rl)
        off = np.abs(np.where(fin, got, 0) - np.where(fin, rl, 0))
        np.testing.assert_array_equal(np.where(fin, 0, got), np.where(fin, 0, rl))
        # the terms P (log P - log q): P and both logarithms
        tol = (kd * tau * tau * 2 + ce) * _log_tol(z, tau) + 4 * R * np.abs(rl)
        assert (off <= np.where(fin, tol, 0)).all(), np.argmax(off)
    if dz is not None:
        got = _f64(dz)
        np.testing.assert_array_equal(np.isnan(got), np.isnan(rd))
        # each part is a probability times its weight: bound by the parts, not their difference
        with np.errstate(invalid="ignore", over="ignore"):
            m = np.where(np.isfinite(Z).any(1, keepdims=True), np.max(np.where(np.isnan(Z), -np.inf, Z), axis=1, keepdims=True), 0)
            q = np.exp((Z - m) / tau)
            q /= np.maximum(q.sum(1, keepdims=True), 1e-300)
            p1 = np.exp(Z - m)
            p1 /= np.maximum(p1.sum(1, keepdims=True), 1e-300)
            up = np.abs(scale * (np.ones(len(Z)) if dloss is None else _f64(dloss)))[:, None]
            parts = up * (kd * tau * q + ce * p1)
            tol = U[z.dtype] * np.abs(rd) + R * (2 * parts + np.abs(rd)) + TINY[z.dtype]
            # listed and label entries: P and the one-hot are parts too
            if i is not None and kd:
                for r in range(len(Z)):
                    tol[r, i[r][i[r] >= 0]] += R * up[r] * kd * tau
            if lab is not None and ce:
                ok = lab >= 0
                tol[np.nonzero(ok)[0], lab[ok]] += R * up[ok, 0] * ce
            if rest is not None and kd:
                # P_rest q / q_rest, with q_rest the mass outside the list
                hide = Z.copy()
                for r in range(len(Z)):
                    hide[r, i[r][i[r] >= 0]] = -np.inf
                hm = np.maximum(hide.max(1, keepdims=True), -1e300)
                qr = np.exp((hide - hm) / tau)
                tol += R * up * kd * tau * 2 * qr / np.maximum(qr.sum(1, keepdims=True), 1e-300)
        tol = np.nan_to_num(tol)  # rows whose logits are NaN and not looked at: exact zeros
        fin = np.isfinite(rd)
        bad = fin & ~(np.abs(got - rd) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0], got[bad][0], rd[bad][0], tol[bad][0])


VS = [(3, 1), (3, 2), (4, 7), (5, 33), (4, 1000), (7, 4097), (3, 32000), (2, 50011), (310, 300)]


@pytest.mark.parametrize("N,V", VS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tau,kd,ce,with_rest", [(1.0, 1.0, 0.0, False), (2.0, 0.7, 0.3, True), (0.5, 1.0, 0.0, True),
                                                 (1.0, 0.4, 0.6, False)])
def test_distill_matches_oracle(N, V, dtype, tau, kd, ce, with_rest):
    rng = np.random.default_rng(N * 1000 + V)
    K = min(V, 17)
    z = _logits(rng, N, V, dtype)
    idx, val = _teacher(rng, z, K)
    rest = torch.from_numpy(rng.normal(1, 1, N).astype(np.float32)).cuda() if with_rest and V > K else None
    lab = rng.integers(0, V, N)
    lab[0] = int(idx[0, 0])
    lab[-1] = -1
    labels = torch.from_numpy(lab.astype(np.int32)).cuda() if ce else None
    dloss = torch.from_numpy(rng.uniform(0.5, 1.5, N).astype(np.float32)).cuda()
    scale = 64.0 if dtype == F16 else 1.0
    op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=tau, kd_weight=kd, ce_weight=ce)
    loss, dz = op.forward_backward(z, idx, val, rest=rest, labels=labels, dloss=dloss, scale=scale)
    torch.cuda.synchronize()
    tw.raise_if_device_error(op.status)
    _check_distill(loss, dz, z, idx, val, rest, labels, tau, kd, ce, dloss, scale)
    # each half alone gives the same bits
    l2, d2 = loss.clone(), dz.clone()
    assert torch.equal(op.forward(z, idx, val, rest=rest, labels=labels), l2)
    dz.zero_()
    assert torch.equal(op.backward(z, idx, val, rest=rest, labels=labels, dloss=dloss, scale=scale), d2)


@pytest.mark.parametrize("dtype,V,N", [(F32, 131071, 2), (BF16, 262144, 2), (F32, 393216, 1), (F16, 100003, 30),
                                       (BF16, 60000, 200), (BF16, 100003, 170), (F32, 60011, 160), (F16, 4099, 400),
                                       (F32, 131070, 153), (BF16, 8191, 2500), (F32, 13001, 320), (F16, 26000, 305)])
def test_distill_long_rows_and_many(dtype, V, N):
    """Sizes on both sides of the choice between a cluster and one CTA a row, and of the
    latter's sizes; more rows than CTAs stay."""
    rng = np.random.default_rng(V)
    K = 64
    z = _logits(rng, N, V, dtype)
    idx, val = _teacher(rng, z, K)
    rest = torch.from_numpy(rng.normal(1, 1, N).astype(np.float32)).cuda()
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=2.0, kd_weight=0.5, ce_weight=0.5)
    loss, dz = op.forward_backward(z, idx, val, rest=rest, labels=labels, scale=256.0)
    _check_distill(loss, dz, z, idx, val, rest, labels, 2.0, 0.5, 0.5, None, 256.0)


@pytest.mark.parametrize("K", [1, 128, 1024])
def test_distill_list_lengths_and_teacher_types(K):
    rng = np.random.default_rng(K)
    z = _logits(rng, 4, 5000, F32)
    idx, val = _teacher(rng, z, K)
    for vt in (F32, BF16, F16):
        op = tw.DistillLoss(4, 5000, K, dtype=F32, temperature=1.3)
        loss, dz = op.forward_backward(z, idx, val.to(vt))
        _check_distill(loss, dz, z, idx, val.to(vt), None, None, 1.3, 1.0, 0.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,off,out_pad", [(5, 0, 5), (0, 3, 0), (3, 1, 4), (8, 8, 16)])
@pytest.mark.parametrize("N", [9, 310, 2500])
def test_distill_strided_rows_write_their_own_columns_only(dtype, pad, off, out_pad, N):
    rng = np.random.default_rng(pad + off)
    V, K = 1237, 5
    z = _logits(rng, N, V, dtype, pad, off)
    idx, val = _teacher(rng, z, K)
    buf = torch.full((N, V + out_pad + off), 9.0, dtype=dtype, device="cuda")
    out = buf[:, off:off + V]
    op = tw.DistillLoss(N, V, K, dtype=dtype, grad=False)
    loss, dz = op.forward_backward(z, idx, val, out=out)
    _check_distill(loss, dz, z, idx, val, None, None, 1.0, 1.0, 0.0)
    assert (buf[:, :off] == 9).all() and (buf[:, off + V:] == 9).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,V", [(9, 1), (9, 2), (9, 9), (9, 17), (9, 1237), (160, 1237), (310, 33), (310, 4099), (2500, 7), (2500, 515),
                                 (9, 90001), (155, 40001)])
def test_distill_gradient_of_rows_aligned_otherwise(dtype, N, V):
    """The alignment of the gradient's rows changes none of its bits, and nothing beside them."""
    rng = np.random.default_rng(V + N)
    K = min(V, 6)
    z = _logits(rng, N, V, dtype, pad=(8 - V) % 8)  # rows on 16 bytes
    idx, val = _teacher(rng, z, K)
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=2.0, kd_weight=0.5, ce_weight=0.5)

    def run(zz, pad, off):
        buf = torch.full((N, off + V + pad), 9.0, dtype=dtype, device="cuda")
        loss, dz = op.forward_backward(zz, idx, val, labels=labels, out=buf[:, off:off + V])
        assert (buf[:, :off] == 9).all() and (buf[:, off + V:] == 9).all()
        return loss.clone(), dz

    for off_z in (0, 3):  # rows that begin on 16 bytes, and 3 elements past them
        zz = torch.zeros((N, off_z + V + (16 - V - off_z) % 8), dtype=dtype, device="cuda")[:, off_z:off_z + V]
        zz.copy_(z)
        loss, dz = run(zz, (16 - V - off_z) % 8, off_z)  # as z's own rows
        _check_distill(loss, dz, zz, idx, val, None, labels, 2.0, 0.5, 0.5)
        for pad, off in [(p, o) for p in (0, 1, 5) for o in (0, 1, 2, 3, 6)] if V < 5000 else [(0, 1), (5, 0)]:
            l2, d2 = run(zz, pad, off)
            assert torch.equal(l2, loss) and torch.equal(d2, dz), (off_z, pad, off)


@pytest.mark.parametrize("dtype,V,N", [(BF16, 777, 5), (F32, 90000, 3), (BF16, 777, 500), (F32, 9001, 310), (BF16, 777, 2600), (BF16, 90001, 155)])
def test_distill_gradient_in_place(dtype, V, N):
    rng = np.random.default_rng(1)
    z = _logits(rng, N, V, dtype, 3).contiguous()
    idx, val = _teacher(rng, z, 8)
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    op = tw.DistillLoss(N, V, 8, dtype=dtype, temperature=2.0, kd_weight=0.5, ce_weight=0.5)
    loss, dz = (t.clone() for t in op.forward_backward(z, idx, val, labels=labels))
    l2, d2 = op.forward_backward(z, idx, val, labels=labels, out=z)
    assert d2.data_ptr() == z.data_ptr()
    assert torch.equal(l2, loss) and torch.equal(z, dz)


@pytest.mark.parametrize("dtype,N,V", [(BF16, 170, 130001), (F32, 160, 70003), (F16, 1300, 30011), (F16, 320, 393216)])
@pytest.mark.parametrize("tau,ce", [(1.0, 0.0), (0.8, 0.5), (2.0, 0.5)])
def test_loss_alone_is_the_loss(dtype, N, V, tau, ce):
    """Without a gradient long rows take another path: the same loss, against the formula's on some rows."""
    rng = np.random.default_rng(N)
    K = 40
    z = torch.randn((N, V), device="cuda", dtype=torch.float32, generator=torch.Generator("cuda").manual_seed(N)).mul_(2.5).to(dtype)
    few = torch.tensor([0, 1, 7, N // 2, N - 2, N - 1], device="cuda")
    idx = torch.from_numpy(np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)).cuda()
    idx[1, 5] = -1
    idx[7, 3] = idx[7, 9]
    idx[0, 0], idx[0, 1] = 0, V - 1
    val = torch.from_numpy(rng.normal(0, 2, (N, K)).astype(np.float32)).cuda()
    rest = torch.from_numpy(rng.normal(1, 1, N).astype(np.float32)).cuda()
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    labels[0], labels[1] = V - 1, -1
    op = tw.DistillLoss(N, V, K, dtype=dtype, temperature=tau, kd_weight=0.7, ce_weight=ce, grad=False)
    loss = op.forward(z, idx, val, rest, labels=labels)
    _check_distill(loss[few], None, z[few], idx[few], val[few], rest[few], labels[few] if ce else None, tau, 0.7, ce)
    tw.raise_if_device_error(op.status)


def test_cross_entropy_alone():
    rng = np.random.default_rng(2)
    z = _logits(rng, 40, 3001, BF16)
    lab = rng.integers(-1, 3001, 40).astype(np.int32)
    lab[:3] = (-1, 0, 3000)
    labels = torch.from_numpy(lab).cuda()
    for tau in (1.0, 2.0):  # the temperature belongs to the teacher's part
        loss, dz, st = tw.distill_loss(z, labels=labels, temperature=tau, kd_weight=0.0, ce_weight=1.0)
        tw.raise_if_device_error(st)
        _check_distill(loss, dz, z, None, None, None, labels, tau, 0.0, 1.0)
        ref = torch.nn.functional.cross_entropy(z.double(), labels.long(), ignore_index=-1, reduction="none")
        assert (loss.double() - ref).abs().max().item() <= _log_tol(z, tau)


@pytest.mark.parametrize("N", [3, 310, 2500])
def test_a_token_listed_twice_counts_twice(N):
    rng = np.random.default_rng(3)
    z = _logits(rng, N, 400, F32).contiguous()
    idx, val = _teacher(rng, z, 6, ragged=False)
    idx[0, 3] = idx[0, 1]
    idx[1, :] = idx[1, 0]
    idx[2, 2:] = idx[2, 1]
    z[2, int(idx[2, 1])] = -float("inf")   # and masked
    rest = torch.zeros(N, device="cuda")
    loss, dz, _ = tw.distill_loss(z, idx, val, rest=rest, temperature=1.5)
    _check_distill(loss, dz, z, idx, val, rest, None, 1.5, 1.0, 0.0)


@pytest.mark.parametrize("V,tiles", [(96, 1), (96, 26), (96, 210), (13001, 1), (13001, 26), (40001, 13)])
def test_masked_tokens_empty_rows_and_special_values(V, tiles):
    """-inf logits on and off the list, at the label, everywhere; the whole vocabulary listed
    with a rest; rows without target whose logits are NaN; NaN and +inf rows; teacher entries
    of logit -inf."""
    rng = np.random.default_rng(4)
    N, K = 12, 4
    inf = float("inf")
    z = _logits(rng, N, V, F32).contiguous()
    idx, val = _teacher(rng, z, K, ragged=False)
    lab = rng.integers(0, V, N).astype(np.int32)
    z[0, 50:] = -inf                       # padded vocabulary
    idx[0] = torch.tensor([1, 2, 3, 4])
    lab[0] = 7
    z[1, int(idx[1, 0])] = -inf            # a listed token the student masks: loss +inf
    z[2, int(lab[2])] = -inf               # a masked label: loss +inf
    z[3] = -inf                            # nothing left
    idx[4] = -1
    lab[4] = -1
    z[4] = float("nan")                    # no target: the logits are not looked at
    z[5, 9] = float("nan")
    z[6, 9] = inf
    val[7] = -inf                          # teacher without mass: the label alone
    val[8, 1:] = -inf
    idx[9, 2:] = -1
    z[10] = -inf
    z[10, 5] = 2.0                         # one token left
    lab[10] = 5
    lab[11] = -1
    labels = torch.from_numpy(lab).cuda()
    for rest in (None, torch.from_numpy(np.r_[np.zeros(4), -inf, np.zeros(2), -inf, np.zeros(4)].astype(np.float32)).cuda()):
        for tau, kd, ce in ((1.0, 0.5, 0.5), (2.0, 0.5, 0.5), (2.0, 1.0, 0.0)):
            many = [None if t is None else t.repeat(tiles, *[1] * (t.dim() - 1)) for t in (z, idx, val, rest, labels)]
            loss, dz, st = tw.distill_loss(many[0], many[1], many[2], rest=many[3], labels=many[4], temperature=tau,
                                           kd_weight=kd, ce_weight=ce)
            tw.raise_if_device_error(st)
            _check_distill(loss[:N], dz[:N], z, idx, val, rest, labels, tau, kd, ce)
            for t in range(1, tiles):
                assert torch.equal(loss[:N].nan_to_num(7.0), loss[t * N:t * N + N].nan_to_num(7.0))
                assert torch.equal(dz[:N].nan_to_num(7.0), dz[t * N:t * N + N].nan_to_num(7.0))
    zs = _logits(rng, 2, 4, F32)
    full = torch.tensor([[3, 1, 0, 2]] * 2, dtype=torch.int32, device="cuda")
    rest = torch.tensor([-inf, 0.0], device="cuda")  # row 1: teacher mass where the student has no token
    fv = torch.zeros(2, 4, device="cuda")
    loss, dz, _ = tw.distill_loss(zs, full, fv, rest=rest)
    _check_distill(loss, dz, zs, full, fv, rest, None, 1.0, 1.0, 0.0)
    assert torch.isinf(loss[1]) and torch.isfinite(loss[0])


def test_index_out_of_range_is_reported_and_skipped():
    rng = np.random.default_rng(5)
    z = _logits(rng, 3, 50, F32)
    idx, val = _teacher(rng, z, 3, ragged=False)
    for bad in (50, -2, 1 << 30):
        i2 = idx.clone()
        i2[1, 1] = bad
        loss, dz, st = tw.distill_loss(z, i2, val)
        assert int(st.item()) == _lib.TW_EINVAL
        i2[1, 1] = -1
        _check_distill(loss, dz, z, i2, val, None, None, 1.0, 1.0, 0.0)
        labels = torch.tensor([1, bad, 2], dtype=torch.int32, device="cuda")
        loss, dz, st = tw.distill_loss(z, labels=labels, kd_weight=0.0, ce_weight=1.0)
        assert int(st.item()) == _lib.TW_EINVAL
        labels[1] = -1
        _check_distill(loss, dz, z, None, None, None, labels, 1.0, 0.0, 1.0)
        lp, _, _, _, st = tw.token_logprobs(z, labels.clone().fill_(bad))
        assert int(st.item()) == _lib.TW_EINVAL and not lp.any()


def test_distill_gradient_against_differences_of_the_loss():
    """Along random directions with the fp32 kernel itself; its loss is good to about 1e-6,
    over h = 1e-2 that leaves 1e-4, and the truncation is h^2."""
    rng = np.random.default_rng(6)
    N, V, K, h = 5, 700, 9, 1e-2
    z = _logits(rng, N, V, F32)
    idx, val = _teacher(rng, z, K)
    rest = torch.zeros(N, device="cuda")
    labels = torch.from_numpy(rng.integers(0, V, N).astype(np.int32)).cuda()
    args = dict(idx=idx, val=val, rest=rest, labels=labels, temperature=1.5, kd_weight=0.6, ce_weight=0.4)
    dz = tw.distill_loss(z, **args)[1].double()
    for k in range(4):
        v = torch.from_numpy(rng.normal(size=(N, V)).astype(np.float32)).cuda()
        up, dn = tw.distill_loss(z + h * v, **args)[0], tw.distill_loss(z - h * v, **args)[0]
        num = (up.double() - dn.double()) / (2 * h)
        ref = (dz * v.double()).sum(1)
        assert ((num - ref).abs() <= 1e-3 * (1 + ref.abs())).all(), (num, ref)


# ------------------------------------------------------------------------------ log probabilities

def _check_logprobs(out, z, tokens, K, tau):
    lp, ent, idx, top = out
    rl, re, ri, rt = ends.token_logprobs(_f64(z), tokens.cpu().numpy(), K, tau)
    tol = _log_tol(z, tau)
    V = z.shape[1]
    # entropy: each p log p is off by R of it and p times the logarithm's error
    for got, ref, t in ((lp, rl, tol), (top, rt, tol), (ent, re, (tol + 2 * R) * (2 + math.log(V)))):
        g = _f64(got)
        fin = np.isfinite(ref)
        np.testing.assert_array_equal(np.where(fin, 0, g), np.where(fin, 0, ref))
        assert (np.abs(g[fin] - ref[fin]) <= t + 2.0 ** -22 * np.abs(ref[fin])).all()
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)


@pytest.mark.parametrize("N,V", VS + [(40, 9001), (2, 262144), (200, 60000), (1300, 3001), (2500, 3001)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("K,S,tau", [(0, 1, 1.0), (1, 1, 0.7), (20, 3, 1.0), (128, 2, 2.0)])
def test_logprobs_match_oracle(N, V, dtype, K, S, tau):
    rng = np.random.default_rng(N + V)
    z = _logits(rng, N, V, dtype)
    tok = rng.integers(0, V, (N, S)).astype(np.int32)
    tok[0, 0] = -1
    tokens = torch.from_numpy(tok).cuda()
    op = tw.TokenLogprobs(N, V, n_tokens=S, top_k=K, temperature=tau, dtype=dtype)
    out = op(z, tokens)
    torch.cuda.synchronize()
    tw.raise_if_device_error(op.status)
    _check_logprobs(out, z, tokens, K, tau)


@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two_values", "one_thread", "zeros_of_both_signs"])
@pytest.mark.parametrize("V,K,tiles", [(5000, 7, 1), (33000, 100, 1), (200000, 20, 1), (5000, 7, 900), (5000, 20, 420)])
def test_alternatives_of_hard_rows(kind, V, K, tiles):
    """Rows whose ties or order defeat a threshold: every element equal, sorted both ways
    (each new one larger than all before), two values, the largest all close together,
    and -0 among 0."""
    z = torch.zeros(3, V, device="cuda")
    if kind in ("ascending", "descending"):
        z += torch.linspace(-5, 5, V, device="cuda")
        z = z.flip(1) if kind == "descending" else z
    elif kind == "two_values":
        z[:, ::2] = 1.0
    elif kind == "one_thread":
        z -= torch.rand(V, device="cuda")
        for s in range(0, min(V, 8 * 512 * 40), 8 * 512):
            z[1, s:s + 8] = 3.0
            z[2, s // 2:s // 2 + 4] = 2.0 + s / V
    elif kind == "zeros_of_both_signs":
        z -= 1
        z[:, 1::3] = -0.0
        z[:, 2::3] = 0.0
    z = z.contiguous()
    for dtype in (F32, BF16):
        zt = z.to(dtype)
        tokens = torch.tensor([[0], [V - 1], [V // 2]], dtype=torch.int32, device="cuda")
        op = tw.TokenLogprobs(3 * tiles, V, top_k=K, dtype=dtype)
        out = op(zt.repeat(tiles, 1), tokens.repeat(tiles, 1))
        _check_logprobs([t[:3] for t in out], zt, tokens, K, 1.0)
        assert all(torch.equal(t.view(tiles, 3, -1), t[:3].view(1, 3, -1).expand(tiles, -1, -1)) for t in out)


def test_logprobs_masks_and_special_rows():
    rng = np.random.default_rng(7)
    inf = float("inf")
    for V in (130, 70000):
        z = _logits(rng, 8, V, F32).contiguous()
        z[0, 3:] = -inf                     # fewer tokens left than alternatives
        z[1] = -inf
        z[2, 5] = float("nan")
        z[3, 6] = inf
        z[4] = -inf
        z[4, V - 1] = -1e30
        z[5] = -torch.finfo(F32).max        # masked by the type's lowest value: all equal
        z[6, 1:] = -torch.finfo(F32).max
        tokens = torch.tensor([[0, V - 1]] * 8, dtype=torch.int32, device="cuda")
        for tau in (1.0, 0.5):
            op = tw.TokenLogprobs(8, V, n_tokens=2, top_k=12, temperature=tau, dtype=F32)
            lp, ent, idx, top = op(z, tokens)
            rl, re, ri, rt = ends.token_logprobs(_f64(z), tokens.cpu().numpy(), 12, tau)
            np.testing.assert_array_equal(idx.cpu().numpy(), ri)
            rows = [0, 1, 2, 3, 4, 7]
            tol = R + 2.0 ** -22 * 64
            for got, ref in ((lp, rl), (top, rt), (ent[:, None], re[:, None])):
                g = _f64(got)[rows]
                ref = ref[rows]
                fin = np.isfinite(ref)
                np.testing.assert_array_equal(np.where(fin, 0, g), np.where(fin, 0, ref))
                assert (np.abs(g[fin] - ref[fin]) <= tol * (2 + math.log(V))).all()
            # probabilities under the lowest value: equal ones uniform, beside a real one 0
            assert abs(float(ent[5]) - math.log(V)) <= tol * (2 + math.log(V)) and float(ent[6]) == 0.0
            assert float(lp[6, 0]) == 0.0 and float(lp[6, 1]) <= -1e30


def test_logprobs_strided_rows_fewer_rows_and_no_tokens():
    rng = np.random.default_rng(8)
    z = _logits(rng, 11, 2999, F16, 7, 3)
    op = tw.TokenLogprobs(64, 2999, n_tokens=1, top_k=5, dtype=F16)
    tokens = torch.from_numpy(rng.integers(0, 2999, (11, 1)).astype(np.int32)).cuda()
    out = op(z, tokens)
    assert out[0].shape == (11, 1) and out[2].shape == (11, 5)
    _check_logprobs(out, z, tokens, 5, 1.0)
    lp, ent, idx, top, st = tw.token_logprobs(z, top_k=5)
    assert lp.shape == (11, 0) and torch.equal(idx, out[2]) and torch.equal(ent, out[1])
    one = z[4:5].expand(6, 2999)
    ent2 = tw.token_logprobs(one, top_k=5)[1]
    assert torch.equal(ent2, ent[4].expand(6)) or (ent2 - ent[4]).abs().max() <= 8 * R * math.log(2999)
    assert op(z[:0], tokens[:0])[0].shape == (0, 1)


@pytest.mark.parametrize("N,V", [(3, 131072), (64, 5000), (310, 5000), (2500, 5000), (160, 70000)])
def test_same_bits_every_time_on_another_stream_and_in_a_graph(N, V):
    rng = np.random.default_rng(9)
    z = _logits(rng, N, V, BF16)
    idx, val = _teacher(rng, z, 16)
    tokens = torch.from_numpy(rng.integers(0, V, (N, 1)).astype(np.int32)).cuda()
    dl = tw.DistillLoss(N, V, 16, temperature=2.0)
    lp = tw.TokenLogprobs(N, V, top_k=8)

    def both():
        return (*dl.forward_backward(z, idx, val), *lp(z, tokens))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [t.clone() for t in both()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_row_offsets_past_32_bits():
    """A buffer of more than 2^32 elements: the last rows lie past every 32-bit offset."""
    N, V = 17, 300000
    ld = (1 << 32) // 16 + 64
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * 2 * N * ld:
        pytest.skip("needs about 27 GB")
    buf = torch.empty(N * ld, dtype=BF16, device="cuda")
    z = buf.as_strided((N, V), (ld, 1))
    rng = np.random.default_rng(10)
    rows = _logits(rng, N, V, BF16)
    z.copy_(rows)
    tokens = torch.from_numpy(rng.integers(0, V, (N, 1)).astype(np.int32)).cuda()
    a = tw.TokenLogprobs(N, V, top_k=4)
    want = [t.clone() for t in a(rows, tokens)]
    assert all(torch.equal(x, y) for x, y in zip(want, a(z, tokens)))
    labels = tokens[:, 0].contiguous()
    op = tw.DistillLoss(N, V, 0, kd_weight=0.0, ce_weight=1.0)
    loss, dz = (t.clone() for t in op.forward_backward(rows, labels=labels))
    l2, d2 = op.forward_backward(z, labels=labels, out=z)
    assert torch.equal(l2, loss) and torch.equal(d2, dz)
