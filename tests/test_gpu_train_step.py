"""Embedding, RMS norms, the layer, the loss and the orthogonalised update used together: one
training step of examples/train_step.py against the same model written with torch autograd in
float64 on the same bf16 weights, its update against oracle/updates.py, several steps for
running, and a step captured into a graph."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import activation_sparse_feedforward_gb300 as tw  # noqa: E402
from oracle import updates  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _norm(s, w):
    return s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * w


def _reference(model, tokens, labels, active):
    """Losses and gradients of their mean by autograd in float64, on the model's own side of
    every ReLU (active: which entries it kept, per layer). Where g lies within the bf16 noise of
    its inputs the sides are a toss-up, and one entry adds or drops its whole term of the
    gradient: noise of 4 * 2^-8.5 / sqrt(3), rms, flips 0.2 % of the active entries, sqrt(0.002)
    = 5 % of Wg's gradient. The entries on the other side are checked to lie there."""
    D = torch.float64
    leaf = lambda t: t.detach().to(D).requires_grad_()  # noqa: E731
    layers = [{k: leaf(v) for k, v in l.items()} for l in model.layers]
    nw, E = leaf(model.norm_w), leaf(model.E)
    s = E[tokens.long()] * model.d ** 0.5
    for l, on in zip(layers, active):
        h = _norm(s, l["norm_w"])
        g = h @ l["Wg"].T
        other = g.detach()[(g > 0) != on]  # g is of norm 1: within ten roundings of 2^-8 at most
        assert other.abs().max() <= 10 * 2.0 ** -8 and other.numel() < 0.01 * on.sum()
        s = s + ((g * on) * (h @ l["Wu"].T)) @ l["Wd"]
    z = _norm(s, nw) @ E.T
    lab = labels.long()
    loss = torch.nn.functional.cross_entropy(z, lab.clamp(min=0), reduction="none") * (lab >= 0)
    loss.mean().backward()
    return loss.detach(), dict(E=E.grad, norm_w=nw.grad, layers=[{k: v.grad for k, v in l.items()} for l in layers])


def test_step_matches_autograd(ex):
    T, d, I, V = 192, 256, 704, 1024
    model = ex.Model(T, d, I, V, layers=2)
    tokens, labels = ex.sequence(T, V)
    losses, grads = model.step(tokens, labels)
    torch.cuda.synchronize()
    model.check()
    active = [tw.hybrid_unpack(f.saved)[0] > 0 for f in model.ffns]
    rl, rg = _reference(model, tokens, labels, active)
    # bf16 activations between the operators: each of about ten roundings of 2^-9 of a term's
    # size moves a gradient by that much
    def close(a, b, rel, what):
        e = (a.double() - b).norm().item() / b.norm().item()
        assert e <= rel, (what, e)
    close(losses, rl, 1e-2, "loss")
    close(grads["E"], rg["E"], 3e-2, "E")
    close(grads["norm_w"], rg["norm_w"], 3e-2, "norm_w")
    for n in range(2):
        for k in ("norm_w", "Wg", "Wu", "Wd"):
            close(grads["layers"][n][k], rg["layers"][n][k], 5e-2, f"layer {n} {k}")


def test_update_matches_oracle(ex):
    T, d, I, V = 128, 256, 704, 1024
    model = ex.Model(T, d, I, V, layers=1, decay=0.1)
    tokens, labels = ex.sequence(T, V)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    for _ in range(2):  # the second with momentum
        _, grads = model.step(tokens, labels)
        was = {k: f64(model.layers[0][k]) for k in ex.HIDDEN}
        buf = {k: f64(model.momentum[0][k]) for k in ex.HIDDEN}
        g = {k: f64(grads["layers"][0][k]) for k in ex.HIDDEN}
        model.update(grads, lr=0.1, hidden_lr=0.05)
        torch.cuda.synchronize()
        model.check()
        for k in ex.HIDDEN:
            new, u = updates.momentum(g[k], buf[k], 0.95)
            assert np.abs(f64(model.momentum[0][k]) - new).max() <= 2.0 ** -22 * (np.abs(buf[k]).max() + np.abs(g[k]).max())
            x = updates.newton_schulz(u) * 0.05 * (I / d) ** 0.5
            want = (1 - 0.05 * 0.1) * was[k] - x
            # the update itself to 15 roundings of fp16 (tests/test_gpu_ortho.py), and bf16's of the weight
            err = np.linalg.norm(f64(model.layers[0][k]) - want)
            assert err <= 15 * 2.0 ** -12 * np.linalg.norm(x) + 2.0 ** -8 * np.linalg.norm(want), k


def test_steps_run_and_stay_finite(ex):
    T, d, I, V = 128, 256, 704, 1024
    model = ex.Model(T, d, I, V, layers=2, l1=1e-7)
    tokens, labels = ex.sequence(T, V)
    for _ in range(8):
        losses, grads = model.step(tokens, labels)
        model.update(grads, lr=0.5, hidden_lr=0.02)
    model.check()
    assert torch.isfinite(losses).all()
    for w in [model.E, model.norm_w] + [l[k] for l in model.layers for k in l]:
        assert torch.isfinite(w.float()).all()


def test_operators_of_a_step_captured_together():
    """Embedding, norms both ways and the update in one graph, replayed on other tokens."""
    T, d, V = 700, 512, 300
    gen = torch.Generator(device="cuda").manual_seed(5)
    E = torch.randn(V, d, generator=gen, device="cuda").bfloat16()
    tokens = torch.randint(-1, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.rand(d, generator=gen, device="cuda") + 0.5

    def objects():
        return tw.Embedding(T, V, d, scale=2.0), tw.RMSNorm(T, d, weight_dtype=torch.float32), tw.Orthogonalize(V, d, momentum=0.9)

    def step(ops, buf, out):
        emb, norm, ortho = ops
        y, s = norm.forward(emb.forward(tokens, E), w)
        dx, dw = norm.backward(y, s, w)
        dE = emb.backward(dx, tokens)
        ortho(dE, buf, out=out, scale=-0.1, beta=0.99)
        return y, dw, dE

    captured, eager = objects(), objects()
    bufs = [torch.zeros(V, d, device="cuda") for _ in range(2)]
    outs = [E.clone() for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(captured, bufs[0].clone(), outs[0].clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(captured, bufs[0], outs[0])
    for _ in range(3):
        tokens.copy_(torch.randint(-1, V, (T,), generator=gen, device="cuda", dtype=torch.int32))
        graph.replay()
        want = step(eager, bufs[1], outs[1])
        torch.cuda.synchronize()
        for a, b in zip((*res, bufs[0], outs[0]), (*want, bufs[1], outs[1])):
            assert torch.equal(a, b)
