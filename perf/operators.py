"""Cases that the model-end operators are measured on: layer norm (forward with the
residual add, backward), the distillation loss with its gradient, and log
probabilities of given tokens with entropy and top alternatives.

``own`` selects what ``run`` calls: the plain forms below (elementary torch
operations in 32 bits) or the package's entry points. ``exact`` is the definition in
64 bits, written apart from the plain forms.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one serving step of a few sequences: the residual add and norm before the FFN
        dict(name="norm_fwd_step", op="norm_fwd", T=8, d=2048, type="bf16", wtype="bf16", residual=True),
        # the norm of a training step's 16384 tokens at the FFN's width, fp32 weights
        dict(name="norm_fwd_train", op="norm_fwd", T=16384, d=2048, type="bf16", wtype="f32", residual=True),
        # a ragged batch at an odd width, no residual
        dict(name="norm_fwd_odd", op="norm_fwd", T=4099, d=1027, type="f16", wtype="f16", residual=False),
        # backward of a short fine-tuning batch: latency of the weight gradient's sum over rows
        dict(name="norm_bwd_short", op="norm_bwd", T=77, d=2048, type="bf16", wtype="f32", residual=True),
        # backward of the training step's norm
        dict(name="norm_bwd_train", op="norm_bwd", T=16384, d=2048, type="bf16", wtype="f32", residual=True),
        # backward in fp32 at the largest width of the repository's configurations
        dict(name="norm_bwd_wide", op="norm_bwd", T=8191, d=8192, type="f32", wtype="f32", residual=False),
        # a few positions' loss and gradient: the smallest distillation call
        dict(name="distill_few", op="distill", N=6, V=32000, K=16, type="bf16", mode="both", tau=1.0, ce=False,
             rest=False, pad=0),
        # a training step: temperature, the teacher's unlisted mass, labels mixed in
        dict(name="distill_train", op="distill", N=4096, V=131072, K=64, type="bf16", mode="both", tau=2.0, ce=True,
             rest=True, pad=0),
        # fp32 logits (what the dense product gives) over an odd vocabulary, ragged teacher lists
        dict(name="distill_odd_f32", op="distill", N=1023, V=50011, K=33, type="f32", mode="both", tau=1.5, ce=False,
             rest=True, pad=0),
        # log probabilities of one decoding step with its alternatives
        dict(name="logprobs_step", op="logprobs", N=1, V=131072, K=20, S=1, type="bf16", tau=1.0, pad=0, mask=0.0),
        # scoring prompts: every position's next token, no alternatives kept but the best few
        dict(name="logprobs_score", op="logprobs", N=8192, V=65536, K=5, S=1, type="bf16", tau=1.0, pad=0, mask=0.0),
        # candidate answers under a vocabulary mask, rows of a padded fp16 buffer, odd sizes
        dict(name="logprobs_masked", op="logprobs", N=333, V=100003, K=8, S=4, type="f16", tau=0.7, pad=29, mask=0.6),
    ]


def _log_uniform(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "distill", "logprobs"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind.startswith("norm"):
        d = _log_uniform(rng, 256, 8192)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
            d += 64 if d == 3072 else 0
        T = min(_log_uniform(rng, 1, 16384), (8191 * 8192 * 4) // (d * SIZE[t]))
        return dict(op=kind, T=T, d=d, type=t, wtype=rng.choice([t, "f32"]), residual=rng.random() < 0.5)
    V = _log_uniform(rng, 4096, 200000)
    if rng.random() < 0.5:
        V = (V + 63) // 64 * 64
    N = min(_log_uniform(rng, 1, 4096), (4096 * 131072 * 2) // ((V + 64) * SIZE[t]))
    pad = rng.choice([0, 0, 5, 64])
    tau = rng.choice([1.0, 1.0, 0.8, 2.0])
    if kind == "distill":
        return dict(op=kind, N=N, V=V, K=rng.randint(1, 128), type=t, mode=rng.choice(["both", "both", "loss", "grad"]),
                    tau=tau, ce=rng.random() < 0.5, rest=rng.random() < 0.5, pad=pad)
    return dict(op=kind, N=N, V=V, K=rng.randint(0, 32), S=rng.choice([1, 1, 3]), type=t, tau=tau, pad=pad,
                mask=rng.choice([0.0, 0.0, 0.5]))


# ------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _logits(g, N, V, pad, dtype):
    """Rows of a [N, V + pad] buffer: a spread of a few units, one in 64 tokens raised."""
    z = _randn(g, N, V + pad, dtype=dtype, scale=2.5)
    z.add_((torch.rand(N, V + pad, generator=g, device="cuda", dtype=dtype) < 1.0 / 64).to(dtype), alpha=4.0)
    return z[:, :V]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[c["type"]]
    s = dict(case=c)
    if c["op"].startswith("norm"):
        T, d, wdt = c["T"], c["d"], TYPES[c["wtype"]]
        s["x"] = _randn(g, T, d).mul_(1.5).add_(0.3).to(dt)
        s["w"] = _randn(g, d, scale=0.2).add_(1.0).to(wdt)
        s["b"] = _randn(g, d, scale=0.1).to(wdt)
        if c["op"] == "norm_fwd":
            s["res"] = _randn(g, T, d, scale=2.0).to(dt) if c["residual"] else None
        else:
            s["dy"] = _randn(g, T, d, scale=0.1).to(dt)
            s["dres"] = _randn(g, T, d, scale=0.1).to(dt) if c["residual"] else None
            x = s["x"].float()
            mean = x.sum(1) / d
            s["mean"], s["rstd"] = mean, (((x - mean[:, None]) ** 2).sum(1) / d + EPS) ** -0.5
        if own:
            import activation_sparse_feedforward_gb300 as tw
            s["op"] = tw.LayerNorm(T, d, dtype=dt, weight_dtype=wdt, eps=EPS)
        return s
    N, V, K = c["N"], c["V"], c["K"]
    s["z"] = _logits(g, N, V, c["pad"], dt)
    if c["op"] == "distill":
        # the teacher agrees with the student up to noise; its list is its top K
        t = s["z"] + _randn(g, N, V, dtype=dt)
        val, idx = torch.topk(t, K, dim=1)
        if c["rest"]:
            rest = torch.empty(N, device="cuda")
            for n in range(0, N, 256):
                u = t[n:n + 256].float().scatter(1, idx[n:n + 256], -math.inf)
                rest[n:n + 256] = torch.logsumexp(u / c["tau"], 1)
            s["rest"] = rest
        else:
            s["rest"] = None
        del t
        # ragged lists: a fifth of the rows keep only a part, a few rows nothing
        keep = torch.where(torch.rand(N, generator=g, device="cuda") < 0.2,
                           torch.randint(0, K + 1, (N,), generator=g, device="cuda"), K)
        s["idx"] = torch.where(torch.arange(K, device="cuda")[None] < keep[:, None], idx, -1).to(torch.int32)
        s["val"] = val.float()
        lab = torch.randint(0, V, (N,), generator=g, device="cuda")
        lab = torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, idx[:, 0], lab)
        lab = torch.where(torch.rand(N, generator=g, device="cuda") < 0.05, -1, lab)
        s["labels"] = lab.to(torch.int32) if c["ce"] else None
        s["dloss"] = torch.rand(N, generator=g, device="cuda") + 0.5
        # the mean over rows; fp16 gradients carry a loss scale so that they do not underflow
        s["scale"] = (2.0 ** 15 if c["type"] == "f16" else 1.0) / N
        if own:
            import activation_sparse_feedforward_gb300 as tw
            s["op"] = tw.DistillLoss(N, V, K, dtype=dt, temperature=c["tau"], kd_weight=0.7 if c["ce"] else 1.0,
                                     ce_weight=0.3 if c["ce"] else 0.0, grad=c["mode"] != "loss")
        return s
    if c["mask"]:
        s["z"].masked_fill_(torch.rand(V, generator=g, device="cuda")[None] < c["mask"], -math.inf)
    s["tokens"] = torch.randint(0, V, (N, c["S"]), generator=g, device="cuda").to(torch.int32)
    if own:
        import activation_sparse_feedforward_gb300 as tw
        s["op"] = tw.TokenLogprobs(N, V, n_tokens=c["S"], top_k=K, temperature=c["tau"], dtype=dt)
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_norm_fwd(s):
    x, d = s["x"].float(), s["case"]["d"]
    total = None
    if s["res"] is not None:
        total = (x + s["res"].float()).to(s["x"].dtype)
        x = total.float()
    mean = x.sum(1) / d
    xc = x - mean[:, None]
    rstd = ((xc * xc).sum(1) / d + EPS) ** -0.5
    y = (xc * rstd[:, None] * s["w"].float() + s["b"].float()).to(s["x"].dtype)
    return dict(y=y, sum=total, mean=mean, rstd=rstd)


def _plain_norm_bwd(s):
    d, dy = s["case"]["d"], s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    gw = dy * s["w"].float()
    c1 = gw.sum(1, keepdim=True) / d
    c2 = (gw * xh).sum(1, keepdim=True) / d
    dx = s["rstd"][:, None] * (gw - c1 - xh * c2)
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0), dbias=dy.sum(0))


def _weights(c):
    return (0.7, 0.3) if c["ce"] else (1.0, 0.0)


def _plain_distill(s):
    c, tau = s["case"], s["case"]["tau"]
    kd_w, ce_w = _weights(c)
    N, V = s["z"].shape
    z, rows = s["z"].float(), torch.arange(N, device="cuda")
    valid = s["idx"] >= 0
    slot = torch.where(valid, s["idx"], V).long()       # padding goes to a column of its own
    # teacher: softmax over the list and the rest
    t = torch.where(valid, s["val"] / tau, -math.inf)
    if s["rest"] is not None:
        t = torch.cat([t, s["rest"][:, None]], 1)
    some = (t > -math.inf).any(1)
    tm = torch.where(some, t.max(1).values, 0.0)
    te = torch.exp(t - tm[:, None])
    ts = torch.where(some, te.sum(1), 1.0)
    P = te / ts[:, None]
    logP = t - tm[:, None] - torch.log(ts)[:, None]
    # student
    zt = z / tau
    m = zt.max(1).values
    e = torch.exp(zt - m[:, None])
    total = e.sum(1)
    logq = zt - m[:, None] - torch.log(total)[:, None]
    at = torch.cat([logq, torch.zeros(N, 1, device="cuda")], 1)[rows[:, None], slot]
    listed_ = torch.zeros(N, V + 1, dtype=torch.bool, device="cuda")
    listed_[rows[:, None], slot] = True
    listed_ = listed_[:, :V]
    if s["rest"] is not None:
        es = (e * ~listed_).sum(1)
        at = torch.cat([at, (torch.log(es) - torch.log(total))[:, None]], 1)
    kd = torch.where(P > 0, P * (logP - at), 0.0).sum(1) * tau * tau
    loss = kd_w * kd
    if ce_w:
        lab = s["labels"].long()
        has = lab >= 0
        m1 = z.max(1).values
        e1 = torch.exp(z - m1[:, None])
        s1 = e1.sum(1)
        ce = torch.log(s1) - (z[rows, lab.clamp(min=0)] - m1)
        loss = loss + ce_w * torch.where(has, ce, 0.0)
    out = {} if c["mode"] == "grad" else dict(loss=loss)
    if c["mode"] == "loss":
        return out
    q = e / total[:, None]
    pt = torch.zeros(N, V + 1, device="cuda")
    pt[rows[:, None], slot] = P[:, :s["idx"].shape[1]]
    pt = pt[:, :V]
    if s["rest"] is not None:
        pt = pt + torch.where(listed_, 0.0, e) * (P[:, -1] / es)[:, None]
    dz = kd_w * tau * (q * some[:, None] - pt)
    if ce_w:
        p1 = e1 / s1[:, None]
        p1[rows, lab.clamp(min=0)] -= 1.0
        dz = dz + ce_w * torch.where(has[:, None], p1, 0.0)
    out["dz"] = (dz * (s["dloss"] * s["scale"])[:, None]).to(s["z"].dtype)
    return out


def _plain_logprobs(s):
    c = s["case"]
    z = s["z"].float()
    N, V = z.shape
    zt = z / c["tau"]
    m = zt.max(1).values
    e = torch.exp(zt - m[:, None])
    total = e.sum(1)
    logp = zt - m[:, None] - torch.log(total)[:, None]
    p = e / total[:, None]
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    rows = torch.arange(N, device="cuda")[:, None]
    out = dict(logprob=logp[rows, s["tokens"].long()], entropy=entropy)
    if c["K"]:
        # ties to the lowest index: unique whole keys, the value's order above the index
        bits = (z + 0.0).view(torch.int32)               # -0.0 ties with 0.0
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = order * (1 << 20) - torch.arange(V, device="cuda")[None]
        idx = torch.topk(key, c["K"], dim=1).indices
        out["top_idx"], out["top_logprob"] = idx.to(torch.int32), logp[rows, idx]
    return out


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "distill": _plain_distill,
                "logprobs": _plain_logprobs}[c["op"]](s)
    op = s["op"]
    if c["op"] == "norm_fwd":
        y, total = op.forward(s["x"], s["w"], s["b"], residual=s["res"])
        return dict(y=y, sum=total if s["res"] is not None else None, mean=op.mean, rstd=op.rstd)
    if c["op"] == "norm_bwd":
        dx, dw, db = op.backward(s["dy"], s["x"], s["w"], dres=s["dres"], mean=s["mean"], rstd=s["rstd"])
        return dict(dx=dx, dweight=dw, dbias=db)
    if c["op"] == "distill":
        if c["mode"] == "loss":
            return dict(loss=op.forward(s["z"], s["idx"], s["val"], rest=s["rest"], labels=s["labels"]))
        if c["mode"] == "grad":
            return dict(dz=op.backward(s["z"], s["idx"], s["val"], rest=s["rest"], labels=s["labels"],
                                       dloss=s["dloss"], scale=s["scale"]))
        loss, dz = op.forward_backward(s["z"], s["idx"], s["val"], rest=s["rest"], labels=s["labels"],
                                       dloss=s["dloss"], scale=s["scale"])
        return dict(loss=loss, dz=dz)
    logprob, entropy, top_idx, top_logprob = op(s["z"], s["tokens"])
    out = dict(logprob=logprob, entropy=entropy)
    if c["K"]:
        out["top_idx"], out["top_logprob"] = top_idx, top_logprob
    return out


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    es = SIZE[c["type"]]
    if c["op"].startswith("norm"):
        T, d, ws = c["T"], c["d"], SIZE[c["wtype"]]
        if c["op"] == "norm_fwd":
            return dict(bytes=T * d * es * (4 if c["residual"] else 2) + 2 * d * ws + 8 * T, flops=8 * T * d)
        return dict(bytes=T * d * es * (4 if c["residual"] else 3) + d * ws + 8 * d + 8 * T, flops=14 * T * d)
    N, V, K = c["N"], c["V"], c["K"]
    if c["op"] == "distill":
        moved = N * V * es * (1 if c["mode"] == "loss" else 2)
        small = N * K * 8 + 4 * N * (bool(c["rest"]) + bool(c["ce"]) + (c["mode"] != "grad") + (c["mode"] != "loss"))
        two = 2 if c["ce"] and c["tau"] != 1.0 else 1
        return dict(bytes=moved + small, flops=N * V * two * (4 if c["mode"] == "loss" else 8))
    return dict(bytes=N * V * es + N * (c["S"] * 8 + 4 + K * 8), flops=6 * N * V)


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    if c["op"] == "norm_fwd":
        total = None
        if s["res"] is not None:
            total = (x + s["res"].double()).to(s["x"].dtype)     # the stored stream is what is normalised
            x = total.double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double())
        return dict(y=y, sum=None if total is None else total.double(), mean=mean, rstd=rstd)
    mean, rstd = s["mean"].double(), s["rstd"].double()
    dy = s["dy"].double()
    xh = (x - mean[:, None]) * rstd[:, None]
    gx = dy * s["w"].double()
    dx = (gx - gx.mean(1, keepdim=True) - xh * (gx * xh).mean(1, keepdim=True)) * rstd[:, None]
    if s["dres"] is not None:
        dx += s["dres"].double()
    return dict(dx=dx, dweight=torch.einsum("td,td->d", dy, xh), dbias=dy.sum(0))


def _exact_distill_row_block(s, a, b, dz):
    c, tau = s["case"], s["case"]["tau"]
    kd_w, ce_w = _weights(c)
    z = s["z"][a:b].double()
    V = z.shape[1]
    logq = torch.log_softmax(z / tau, 1)
    idx, val = s["idx"][a:b].long(), s["val"][a:b].double() / tau
    val = val.masked_fill(idx < 0, -math.inf)
    logq_rest, t = None, val
    if s["rest"] is not None:
        hide = torch.zeros(b - a, V + 1, device="cuda", dtype=torch.float64)
        hide.scatter_(1, idx.masked_fill(idx < 0, V), -math.inf)
        unlisted = logq + hide[:, :V]
        del hide
        logq_rest = torch.logsumexp(unlisted, 1)
        t = torch.cat([val, s["rest"][a:b].double()[:, None]], 1)
    lse = torch.logsumexp(t, 1, keepdim=True)
    empty = torch.isneginf(lse)
    logP = t - lse.masked_fill(empty, 0.0)
    P = torch.exp(logP)
    other = torch.gather(logq, 1, idx.clamp(min=0))
    if logq_rest is not None:
        other = torch.cat([other, logq_rest[:, None]], 1)
    term = (P * (logP - other)).masked_fill(P == 0, 0.0)
    loss = kd_w * tau ** 2 * term.sum(1)
    has = None
    if ce_w:
        lab = s["labels"][a:b].long()
        has = lab >= 0
        lp = torch.log_softmax(z, 1)
        loss = loss - ce_w * torch.gather(lp, 1, lab.clamp(min=0)[:, None])[:, 0].masked_fill(~has, 0.0)
    if dz is not None:
        gr = torch.exp(logq).masked_fill(empty, 0.0)
        if logq_rest is not None:
            gr -= torch.exp(unlisted + (logP[:, -1] - logq_rest)[:, None])
        gr.scatter_add_(1, idx.clamp(min=0), -P[:, :idx.shape[1]])
        gr *= kd_w * tau
        if ce_w:
            p1 = torch.exp(lp)
            p1.scatter_add_(1, lab.clamp(min=0)[:, None], torch.full((b - a, 1), -1.0, device="cuda", dtype=torch.float64))
            gr += ce_w * p1.masked_fill(~has[:, None], 0.0)
        dz[a:b] = gr * (s["dloss"][a:b].double() * s["scale"])[:, None]
    return loss


def _exact_logprobs(s):
    c = s["case"]
    lps, ents, tops = [], [], []
    for n in range(0, c["N"], 512):
        z = s["z"][n:n + 512].double()
        lp = torch.log_softmax(z / c["tau"], 1)
        lps.append(torch.gather(lp, 1, s["tokens"][n:n + 512].long()))
        ents.append(torch.special.entr(torch.exp(lp)).sum(1))
        if c["K"]:
            tops.append(torch.topk(lp, c["K"], 1).values)
    out = dict(logprob=torch.cat(lps), entropy=torch.cat(ents))
    if c["K"]:
        out["top_idx"], out["top_logprob"] = None, torch.cat(tops)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    N, V = case["N"], case["V"]
    dz = torch.empty(N, V, device="cuda", dtype=torch.float64) if case["mode"] != "loss" else None
    loss = torch.cat([_exact_distill_row_block(s, n, min(n + 256, N), dz) for n in range(0, N, 256)])
    out = {} if case["mode"] == "grad" else dict(loss=loss)
    if dz is not None:
        out["dz"] = dz
    return out
