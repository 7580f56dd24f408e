"""Training a small ReLU-sparse residual model from a teacher's top logits, and scoring it.

    h_0 = x;   h_{l+1} = h_l + FFN_l(norm_l(h_l));   logits = norm(h_L) E^T

Each layer's feedforward runs through the Hybrid format (forward, backward, L1 penalty);
the residual adds, norms and their gradients are the layer-norm operator's; the loss is
the distillation loss with hard labels mixed in; the read-out is the token log
probabilities. Every step runs in the library's kernels except the optimiser's update and
the casts between them. Shapes: FFN widths as HybridFFN wants them, vocabulary % 64 == 0.

    python examples/distill_step.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_feedforward_gb300 as tw

BF16, F32 = torch.bfloat16, torch.float32


class Model:
    """Weights, their gradients and the operators' buffers for T tokens."""

    def __init__(self, T: int, d: int, I: int, V: int, layers: int, K: int, temperature: float = 2.0,
                 kd_weight: float = 0.7, ce_weight: float = 0.3, l1: float = 0.0, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.V, self.l1 = T, d, V, l1

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        self.layers = [dict(norm_w=torch.ones(d, device="cuda"), norm_b=torch.zeros(d, device="cuda"),
                            Wg=normal(I, d, std=d ** -0.5), Wu=normal(I, d, std=d ** -0.5),
                            Wd=normal(I, d, std=I ** -0.5)) for _ in range(layers)]
        self.norm_w, self.norm_b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
        self.E = normal(V, d, std=d ** -0.5)
        self.norms = [tw.LayerNorm(T, d, weight_dtype=F32) for _ in range(layers + 1)]
        self.ffns = [tw.HybridFFN(T, d, I, W=64, C=64, R=I, backup_cap=0, gated=True) for _ in range(layers)]
        self.loss = tw.DistillLoss(T, V, K, dtype=F32, temperature=temperature, kd_weight=kd_weight,
                                   ce_weight=ce_weight, grad=False)
        self.status = tw.new_status()

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        """fp32 [T, V]. A layer's feedforward output is the next norm's x, the stream its
        residual, so the add and the norm are one pass."""
        stream, out = x, None
        self.inputs, self.streams = [], []
        for layer, norm, ffn in zip(self.layers, self.norms, self.ffns):
            h, stream = norm.forward(stream if out is None else out, layer["norm_w"], layer["norm_b"],
                                     residual=None if out is None else stream)
            self.inputs.append(h)
            self.streams.append(stream)
            out = ffn.forward(h, layer["Wg"], layer["Wu"], layer["Wd"])
        h, stream = self.norms[-1].forward(out, self.norm_w, self.norm_b, residual=stream)
        self.inputs.append(h)
        self.streams.append(stream)
        return tw.dense_gemm(h, self.E, self.T, self.V, self.d, False, False, status=self.status)

    def step(self, x, idx, val, rest=None, labels=None):
        """Losses [T] and the gradients of every weight for the mean loss (plus l1 * the
        activations' sum)."""
        z = self.logits(x)
        losses, dz = self.loss.forward_backward(z, idx, val, rest=rest, labels=labels, scale=1.0 / self.T, out=z)
        dz = dz.to(BF16)
        dh = tw.dense_gemm(dz, self.E, self.T, self.d, self.V, False, True, status=self.status).to(BF16)
        grads = dict(E=tw.dense_gemm(dz, self.inputs[-1], self.V, self.d, self.T, True, True, status=self.status))
        stream_grad, grads["norm_w"], grads["norm_b"] = self.norms[-1].backward(dh, self.streams[-1], self.norm_w)
        grads["layers"] = [None] * len(self.layers)
        for n in reversed(range(len(self.layers))):
            layer = self.layers[n]
            dh, dWg, dWu, dWd = self.ffns[n].backward(stream_grad, self.inputs[n], layer["Wg"], layer["Wu"], layer["Wd"],
                                                      l1=self.l1)
            # what reaches the stream: through the norm, and past the block
            stream_grad, dw, db = self.norms[n].backward(dh, self.streams[n], layer["norm_w"], dres=stream_grad)
            grads["layers"][n] = dict(norm_w=dw, norm_b=db, Wg=dWg, Wu=dWu, Wd=dWd)
        return losses, grads

    def update(self, grads, lr: float) -> None:
        """Plain gradient descent, in place."""
        pairs = [(self.E, grads["E"]), (self.norm_w, grads["norm_w"]), (self.norm_b, grads["norm_b"])]
        for layer, g in zip(self.layers, grads["layers"]):
            pairs += [(layer[k], g[k]) for k in g]
        for w, g in pairs:
            w.sub_((lr * g).to(w.dtype))

    def check(self) -> None:
        """Raises what the device reported (synchronises)."""
        for where, s in [("product", self.status), ("loss", self.loss.status)] + [("ffn", f.status) for f in self.ffns]:
            tw.raise_if_device_error(s, where)


def teacher_targets(T: int, V: int, K: int, temperature: float, seed: int = 1):
    """A synthetic teacher: peaked logits, their top K, the rest's mass, its argmax as label."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(T, V, generator=g, device="cuda") * 2
    val, idx = torch.topk(t, K, dim=1)
    rest = torch.logsumexp(t.scatter(1, idx, float("-inf")) / temperature, 1)
    return idx.int(), val.contiguous(), rest, idx[:, 0].int().contiguous()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    T, d, I, V, K, tau = a.tokens, 512, 1408, 4096, 32, 2.0
    model = Model(T, d, I, V, layers=2, K=K, temperature=tau, l1=1e-7)
    x = torch.randn(T, d, device="cuda").to(BF16)
    idx, val, rest, labels = teacher_targets(T, V, K, tau)
    score = tw.TokenLogprobs(T, V, n_tokens=1, top_k=3, dtype=F32)
    for n in range(a.steps):
        losses, grads = model.step(x, idx, val, rest, labels)
        model.update(grads, lr=4.0)
        if n % 5 == 0 or n == a.steps - 1:
            mean = losses.mean().item()
            logprob, entropy, top, _ = score(model.logits(x), labels)
            hit = (top[:, 0] == labels).float().mean().item()
            print(f"step {n:3d}  loss {mean:.4f}  label log probability {logprob.mean().item():.3f}  "
                  f"entropy {entropy.mean().item():.3f}  top-1 agreement {hit:.3f}")
    model.check()


if __name__ == "__main__":
    main()
