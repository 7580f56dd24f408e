"""The operators used together: one training step of examples/distill_step.py against the
same model written with torch autograd in float64 on the same bf16 weights, and a few
steps that have to lower the loss."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location("distill_step", os.path.join(ROOT, "examples", "distill_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(model, x, idx, val, rest, labels, tau, kd, ce):
    """Mean loss and gradients by autograd in float64."""
    D = torch.float64
    leaf = lambda t: t.detach().to(D).requires_grad_()  # noqa: E731
    layers = [{k: leaf(v) for k, v in l.items()} for l in model.layers]
    nw, nb, E = leaf(model.norm_w), leaf(model.norm_b), leaf(model.E)
    s = x.to(D)
    for l in layers:
        h = torch.nn.functional.layer_norm(s, (s.shape[1],), l["norm_w"], l["norm_b"], 1e-5)
        s = s + (torch.relu(h @ l["Wg"].T) * (h @ l["Wu"].T)) @ l["Wd"]
    z = torch.nn.functional.layer_norm(s, (s.shape[1],), nw, nb, 1e-5) @ E.T
    P = torch.softmax(torch.cat([val.to(D) / tau, rest.to(D)[:, None]], 1), 1)
    lq = torch.log_softmax(z / tau, 1)
    li = idx.long()
    lr = torch.logsumexp(lq.masked_fill(torch.zeros_like(lq, dtype=torch.bool).scatter(1, li, True), -float("inf")), 1)
    kl = (P * (P.log() - torch.cat([lq.gather(1, li), lr[:, None]], 1))).sum(1)
    loss = kd * tau * tau * kl + ce * torch.nn.functional.cross_entropy(z, labels.long(), reduction="none")
    loss.mean().backward()
    return loss.detach(), dict(E=E.grad, norm_w=nw.grad, norm_b=nb.grad,
                               layers=[{k: v.grad for k, v in l.items()} for l in layers])


def test_step_matches_autograd(ex):
    T, d, I, V, K, tau = 192, 256, 704, 1024, 16, 2.0
    model = ex.Model(T, d, I, V, layers=2, K=K, temperature=tau)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    idx, val, rest, labels = ex.teacher_targets(T, V, K, tau)
    losses, grads = model.step(x, idx, val, rest, labels)
    torch.cuda.synchronize()
    model.check()
    rl, rg = _reference(model, x, idx, val, rest, labels, tau, 0.7, 0.3)
    # bf16 activations between the operators: each of about ten roundings of 2^-9 of a
    # term's size moves a gradient by that much, a few per cent in all where signs differ
    def close(a, b, rel, what):
        e = (a.double() - b).norm().item() / b.norm().item()
        assert e <= rel, (what, e)
    close(losses, rl, 1e-2, "loss")
    close(grads["E"], rg["E"], 3e-2, "E")
    close(grads["norm_w"], rg["norm_w"], 3e-2, "norm_w")
    close(grads["norm_b"], rg["norm_b"], 3e-2, "norm_b")
    for n in range(2):
        for k in ("norm_w", "norm_b", "Wg", "Wu", "Wd"):
            close(grads["layers"][n][k], rg["layers"][n][k], 5e-2, f"layer {n} {k}")


def test_steps_lower_the_loss(ex):
    T, d, I, V, K, tau = 128, 256, 704, 1024, 16, 2.0
    model = ex.Model(T, d, I, V, layers=1, K=K, temperature=tau)
    x = torch.randn(T, d, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    targets = ex.teacher_targets(T, V, K, tau)
    first = None
    for _ in range(12):
        losses, grads = model.step(x, *targets)
        first = losses.mean().item() if first is None else first
        model.update(grads, lr=4.0)
    model.check()
    assert losses.mean().item() < 0.8 * first
