"""Cases that the operators of a training step around the feedforward layer are measured on:
the token embedding with its gradient, root-mean-square norm (forward with the residual add,
into 16 bits or into 8 with scales; backward), and the orthogonalised update of hidden weight
matrices (momentum and Newton-Schulz products).

``own`` selects what ``run`` calls: the plain forms below (elementary torch operations in
32 bits) or the package's entry points. ``exact`` is the definition in 64 bits, written apart
from the plain forms.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
STEPS, COEFFICIENTS = 5, (3.4445, -4.7750, 2.0315)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
FP8_MAX, FP8_LEAST_SCALE = 448.0, 2.0 ** -126


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the tokens of one serving step of a few sequences
        dict(name="embed_step", op="embed", T=8, V=131072, d=2048, type="bf16", wtype="bf16", scale=45.25),
        # a training step's 16384 tokens, the table kept in 32 bits
        dict(name="embed_train", op="embed", T=16384, V=131072, d=2048, type="bf16", wtype="f32", scale=1.0),
        # a short fine-tuning batch, added to the gradient that the tied output matrix left: latency
        dict(name="embed_grad_short", op="embed_grad", T=77, V=32000, d=2048, type="bf16", scale=1.0, add=True),
        # the training step's gradient, written whole
        dict(name="embed_grad_train", op="embed_grad", T=16384, V=131072, d=2048, type="bf16", scale=1.0, add=False),
        # odd sizes, many tokens of a small vocabulary: long runs of one token
        dict(name="embed_grad_odd", op="embed_grad", T=40009, V=5003, d=1027, type="f16", scale=0.5, add=True),
        # one serving step: the norm before an 8-bit product, a scale a row
        dict(name="rms_fp8_step", op="rms", T=8, d=2048, type="bf16", wtype="bf16", residual=True, out="fp8", group=0),
        # the training step's norm at the layer's width
        dict(name="rms_train", op="rms", T=16384, d=2048, type="bf16", wtype="f32", residual=True, out="same", group=0),
        # a prefill at the largest hidden width, a scale for each 128 columns, ragged rows
        dict(name="rms_fp8_wide", op="rms", T=8191, d=8192, type="bf16", wtype="bf16", residual=False, out="fp8",
             group=128),
        # backward of the training step's norm with the residual's gradient
        dict(name="rms_grad_train", op="rms_grad", T=16384, d=2048, type="bf16", wtype="f32", residual=True),
        # the smallest layer of this repository's workloads
        dict(name="ortho_small", op="ortho", m=704, n=256, count=1, type="f32", momentum=0.95),
        # the three weight gradients of one layer of a training step, momentum kept in 32 bits
        dict(name="ortho_train", op="ortho", m=5632, n=2048, count=3, type="f32", momentum=0.95),
        # a wide odd matrix of 16-bit gradients, no momentum
        dict(name="ortho_odd", op="ortho", m=1027, n=2500, count=2, type="bf16", momentum=0.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["embed", "embed_grad", "embed_grad", "rms", "rms_grad", "ortho", "ortho"])
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "ortho":
        m, n = _log_uniform(rng, 64, 5632), _log_uniform(rng, 64, 5632)
        if rng.random() < 0.5:
            m, n = (m + 63) // 64 * 64, (n + 63) // 64 * 64
        n, m = (min(n, 2048), m) if n <= m else (n, min(m, 2048))
        return dict(op=kind, m=m, n=n, count=rng.randint(1, 3), type=rng.choice(["f32", "f32", "bf16", "f16"]),
                    momentum=rng.choice([0.0, 0.95]))
    d = _log_uniform(rng, 256, 8192)
    if rng.random() < 0.6:
        d = (d + 63) // 64 * 64
    T = _log_uniform(rng, 1, 40000)
    if kind.startswith("rms"):
        T = min(T, (8191 * 8192 * 2) // (d * SIZE[t]))
        c = dict(op=kind, T=T, d=d, type=t, wtype=rng.choice([t, "f32"]), residual=rng.random() < 0.5)
        if kind == "rms":
            c["out"] = rng.choice(["same", "fp8"])
            c["group"] = rng.choice([0, 128]) if c["out"] == "fp8" else 0
        return c
    T = min(T, (16384 * 2048 * 4) // (d * SIZE[t]))
    V = min(_log_uniform(rng, 1000, 200000), (131072 * 2048) // d)
    c = dict(op=kind, T=T, V=V, d=d, type=t, scale=rng.choice([1.0, 1.0, 0.5, 45.25]))
    if kind == "embed":
        c["wtype"] = rng.choice([t, "f32"])
    else:
        c["add"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _tokens(g, T, V):
    """Frequencies as 1 / rank, the ranks in no order of the indices; one in 50 is padding."""
    rank = torch.exp(torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * math.log(V + 1.0)).long() - 1
    tok = torch.randperm(V, generator=g, device="cuda")[rank.clamp(0, V - 1)]
    return torch.where(torch.rand(T, generator=g, device="cuda") < 0.02, -1, tok).to(torch.int32)


def _gradient(g, m, n, dt):
    """A weight gradient as training gives it: neurons and features of unlike activity, and a
    few directions that many tokens share."""
    rows = torch.exp(_randn(g, m, 1))
    cols = (torch.randperm(n, generator=g, device="cuda") + 1.0)[None] ** -0.5
    shared = (_randn(g, m, 16) * rows) @ (_randn(g, 16, n) * cols)
    return ((_randn(g, m, n) * rows * cols + 0.3 * shared) * 1e-3).to(dt)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[c["type"]]
    s = dict(case=c)
    if c["op"] == "ortho":
        m, n, k = c["m"], c["n"], c["count"]
        s["grads"] = [_gradient(g, m, n, dt) for _ in range(k)]
        s["buffers"] = [_gradient(g, m, n, torch.float32) * 8.0 for _ in range(k)] if c["momentum"] else None
        s["scale"] = max(1.0, m / n) ** 0.5
        if own:
            import activation_sparse_feedforward_gb300 as tw
            s["op"] = tw.Orthogonalize(m, n, count=k, dtype=torch.bfloat16, grad_dtype=dt, steps=STEPS,
                                       momentum=c["momentum"])
        return s
    T, d = c["T"], c["d"]
    if c["op"].startswith("embed"):
        V = c["V"]
        s["tokens"] = _tokens(g, T, V)
        if c["op"] == "embed":
            s["w"] = _randn(g, V, d, dtype=TYPES[c["wtype"]], scale=0.02)
        else:
            s["dy"] = _randn(g, T, d, scale=0.1).to(dt)
            s["dw"] = _randn(g, V, d, scale=0.05) if c["add"] else None
        if own:
            import activation_sparse_feedforward_gb300 as tw
            if c["op"] == "embed":
                s["op"] = tw.Embedding(T, V, d, dtype=dt, weight_dtype=TYPES[c["wtype"]], scale=c["scale"],
                                       backward=False)
            else:
                s["op"] = tw.Embedding(T, V, d, dtype=dt, scale=c["scale"], dweight=not c["add"])
        return s
    wdt = TYPES[c["wtype"]]
    x = _randn(g, T, d, scale=1.5)
    x[:, ::97] *= 12.0                                   # a few channels that stand out
    s["x"] = x.to(dt)
    s["w"] = _randn(g, d, scale=0.2).add_(1.0).to(wdt)
    if c["op"] == "rms":
        s["res"] = _randn(g, T, d, scale=2.0).to(dt) if c["residual"] else None
    else:
        s["dy"] = _randn(g, T, d, scale=0.1).to(dt)
        s["dres"] = _randn(g, T, d, scale=0.1).to(dt) if c["residual"] else None
        x = s["x"].float()
        s["rstd"] = ((x * x).sum(1) / d + EPS) ** -0.5
    if own:
        import activation_sparse_feedforward_gb300 as tw
        s["op"] = tw.RMSNorm(T, d, dtype=dt, weight_dtype=wdt, eps=EPS, backward=c["op"] == "rms_grad",
                             fp8=c.get("out") == "fp8", group=c.get("group", 0))
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_embed(s):
    tok = s["tokens"].long()
    y = s["w"][tok.clamp(min=0)].float() * s["case"]["scale"]
    return dict(y=torch.where(tok[:, None] >= 0, y, 0.0).to(TYPES[s["case"]["type"]]))


def _plain_embed_grad(s):
    c, tok = s["case"], s["tokens"].long()
    dw = s["dw"] if c["add"] else torch.zeros(c["V"], c["d"], device="cuda")
    g = torch.where(tok[:, None] >= 0, s["dy"].float() * c["scale"], 0.0)
    dw.index_add_(0, tok.clamp(min=0), g)
    return dict(dweight=dw)


def _plain_rms(s):
    c, x, d = s["case"], s["x"].float(), s["case"]["d"]
    total = None
    if s["res"] is not None:
        total = (x + s["res"].float()).to(s["x"].dtype)
        x = total.float()
    rstd = ((x * x).sum(1) / d + EPS) ** -0.5
    y = x * rstd[:, None] * s["w"].float()
    out = dict(sum=total, rstd=rstd)
    if c["out"] == "same":
        out["y"] = y.to(s["x"].dtype)
        return out
    group = c["group"] or d
    parts = -(-d // group)
    y = torch.cat([y, torch.zeros(c["T"], parts * group - d, device="cuda")], 1).view(c["T"], parts, group)
    scale = (y.abs().amax(2) / FP8_MAX).clamp(min=FP8_LEAST_SCALE)
    out["q"] = (y / scale[:, :, None]).view(c["T"], -1)[:, :d].to(torch.float8_e4m3fn)
    out["scale"] = scale
    return out


def _plain_rms_grad(s):
    d, dy, r = s["case"]["d"], s["dy"].float(), s["rstd"][:, None]
    xh = s["x"].float() * r
    gw = dy * s["w"].float()
    dx = r * (gw - xh * ((gw * xh).sum(1, keepdim=True) / d))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0))


def _plain_ortho(s):
    c = s["case"]
    x = torch.stack([g.float() for g in s["grads"]])
    if s["buffers"] is not None:
        mu = c["momentum"]
        for buf, g in zip(s["buffers"], x):
            buf.mul_(mu).add_(g)
        x = x + mu * torch.stack(s["buffers"])
    wide = c["m"] < c["n"]
    if wide:
        x = x.transpose(1, 2)
    x = x / (x * x).sum((1, 2), keepdim=True) ** 0.5
    a, b, k = COEFFICIENTS
    for _ in range(STEPS):
        gram = x.transpose(1, 2) @ x
        x = a * x + x @ (b * gram + k * (gram @ gram))
    if wide:
        x = x.transpose(1, 2)
    return dict(out=list((x * s["scale"]).to(torch.bfloat16)), momentum=s["buffers"])


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "rms": _plain_rms, "rms_grad": _plain_rms_grad,
                "ortho": _plain_ortho}[c["op"]](s)
    op = s["op"]
    if c["op"] == "embed":
        return dict(y=op.forward(s["tokens"], s["w"]))
    if c["op"] == "embed_grad":
        return dict(dweight=op.backward(s["dy"], s["tokens"], out=s["dw"], add=c["add"]))
    if c["op"] == "rms":
        if c["out"] == "fp8":
            q, scale, total = op.forward_fp8(s["x"], s["w"], residual=s["res"])
            out = dict(q=q, scale=scale)
        else:
            y, total = op.forward(s["x"], s["w"], residual=s["res"])
            out = dict(y=y)
        return dict(out, sum=total if s["res"] is not None else None, rstd=op.rstd)
    if c["op"] == "rms_grad":
        dx, dw = op.backward(s["dy"], s["x"], s["w"], dres=s["dres"], rstd=s["rstd"])
        return dict(dx=dx, dweight=dw)
    return dict(out=op(s["grads"], s["buffers"], scale=s["scale"]), momentum=s["buffers"])


# ------------------------------------------------------------------------------ what a pass cannot do without

def _distinct(T, V):
    """Expected number of different tokens among T of _tokens' distribution."""
    p = torch.log1p(1.0 / torch.arange(1, V + 1, dtype=torch.float64)) / math.log(V + 1.0)
    return int((1.0 - torch.exp(-0.98 * T * p)).sum())


def work(case):
    c = case
    es = SIZE[c["type"]]
    if c["op"] == "ortho":
        m, n = max(c["m"], c["n"]), min(c["m"], c["n"])
        moved = m * n * (es + 2 + (8 if c["momentum"] else 0))
        # gram and its square are symmetric: half of each product
        return dict(bytes=c["count"] * moved, flops=c["count"] * STEPS * (3 * m * n * n + n ** 3))
    T, d = c["T"], c["d"]
    if c["op"] == "embed":
        return dict(bytes=T * d * es + _distinct(T, c["V"]) * d * SIZE[c["wtype"]] + 4 * T, flops=T * d)
    if c["op"] == "embed_grad":
        rows = 2 * _distinct(T, c["V"]) if c["add"] else c["V"]
        return dict(bytes=T * d * es + rows * d * 4 + 4 * T, flops=2 * T * d)
    ws = SIZE[c["wtype"]]
    if c["op"] == "rms":
        scales = 4 * T * (-(-d // c["group"]) if c["group"] else 1)
        written = T * d + scales if c["out"] == "fp8" else T * d * es
        return dict(bytes=T * d * es * (3 if c["residual"] else 1) + written + d * ws + 4 * T, flops=5 * T * d)
    return dict(bytes=T * d * es * (4 if c["residual"] else 3) + d * ws + 4 * d + 4 * T, flops=10 * T * d)


# ------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_embed(s):
    c = s["case"]
    y = torch.zeros(c["T"], c["d"], device="cuda", dtype=torch.float64)
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    y[at] = torch.index_select(s["w"], 0, s["tokens"][at].long()).double().mul_(c["scale"])
    return dict(y=y)


def _exact_embed_grad(s):
    c = s["case"]
    dw = s["dw"].double() if c["add"] else torch.zeros(c["V"], c["d"], device="cuda", dtype=torch.float64)
    at = torch.nonzero(s["tokens"] >= 0)[:, 0]
    dw.index_add_(0, s["tokens"][at].long(), s["dy"][at].double(), alpha=c["scale"])
    return dict(dweight=dw)


def _exact_rms(s):
    c = s["case"]
    x = s["x"].double()
    total = None
    if s["res"] is not None:
        x = (x + s["res"].double()).to(s["x"].dtype).double()     # the stored stream is what is normalised
        total = x
    rstd = torch.rsqrt(x.square().mean(1) + EPS)
    y = torch.einsum("td,t,d->td", x, rstd, s["w"].double())
    out = dict(sum=total, rstd=rstd)
    if c["out"] == "same":
        return dict(out, y=y)
    scales, qs = [], []
    for part in y.split(c["group"] or c["d"], 1):
        scale = torch.linalg.vector_norm(part, math.inf, 1) / FP8_MAX
        scales.append(scale.clamp(min=FP8_LEAST_SCALE))
        qs.append(part / scales[-1][:, None])
    return dict(out, q=torch.cat(qs, 1), scale=torch.stack(scales, 1))


def _exact_rms_grad(s):
    x, dy, w, r = s["x"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()
    g = dy * w
    along = torch.einsum("td,td->t", g, x) * r ** 3 / x.shape[1]
    dx = g * r[:, None] - x * along[:, None]
    if s["dres"] is not None:
        dx += s["dres"].double()
    return dict(dx=dx, dweight=torch.einsum("td,td,t->d", dy, x, r))


def _exact_ortho(s):
    c = s["case"]
    a, b, k = COEFFICIENTS
    outs, bufs = [], []
    for i, g in enumerate(s["grads"]):
        x = g.double()
        if s["buffers"] is not None:
            bufs.append(torch.add(x, s["buffers"][i].double(), alpha=c["momentum"]))
            x = torch.add(x, bufs[-1], alpha=c["momentum"])
        x = x / torch.linalg.matrix_norm(x)
        tall = x.shape[0] >= x.shape[1]
        for _ in range(STEPS):
            if tall:
                gram = torch.mm(x.T, x)
            else:
                gram = torch.mm(x, x.T)
            p = torch.addmm(gram, gram, gram, beta=b, alpha=k)
            p.diagonal().add_(a)
            x = torch.mm(x, p) if tall else torch.mm(p, x)
        outs.append(x * s["scale"])
    return dict(out=outs, momentum=bufs if bufs else None)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "rms": _exact_rms, "rms_grad": _exact_rms_grad,
            "ortho": _exact_ortho}[case["op"]](s)
