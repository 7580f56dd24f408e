"""Training a small ReLU-sparse language model from tokens: embedding, RMS norms, Hybrid
feedforward layers, tied output matrix, and orthogonalised updates of the hidden matrices.

    s_0 = c E[tokens];   s_{l+1} = s_l + FFN_l(norm_l(s_l));   logits = norm(s_L) E^T

The residual adds, norms and their gradients are the RMS-norm operator's; the output
matrix's gradient is written by a product and the embedding's added to it; the loss is the
distillation loss with labels alone, or with a teacher. Wg, Wu and Wd are updated in place by
their orthogonalised momentum, all three of a layer in one call, the other weights by plain
gradient descent. Shapes: FFN widths as HybridFFN wants them, tokens and vocabulary % 64 == 0.

    python examples/train_step.py [--steps 20]
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
HIDDEN = ("Wg", "Wu", "Wd")


class Model:
    """Weights, momentum and the operators' buffers for T tokens."""

    def __init__(self, T: int, d: int, I: int, V: int, layers: int, l1: float = 0.0, decay: float = 0.01, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.V, self.l1, self.decay = T, d, V, l1, decay

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

        self.layers = [dict(norm_w=torch.ones(d, device="cuda"), Wg=normal(I, d, std=d ** -0.5),
                            Wu=normal(I, d, std=d ** -0.5), Wd=normal(I, d, std=I ** -0.5)) for _ in range(layers)]
        self.momentum = [{k: torch.zeros(I, d, device="cuda") for k in HIDDEN} for _ in range(layers)]
        self.norm_w = torch.ones(d, device="cuda")
        self.E = normal(V, d, std=d ** -0.5)
        # the table's rows are as the output matrix wants them: of norm 1; the stream wants elements of 1
        self.embed = tw.Embedding(T, V, d, scale=d ** 0.5, dweight=False)
        self.norms = [tw.RMSNorm(T, d, weight_dtype=F32) for _ in range(layers + 1)]
        self.ffns = [tw.HybridFFN(T, d, I, W=64, C=64, R=I, backup_cap=0, gated=True) for _ in range(layers)]
        self.loss = tw.DistillLoss(T, V, 0, dtype=F32, kd_weight=0.0, ce_weight=1.0, grad=False)
        self.ortho = tw.Orthogonalize(I, d, count=len(HIDDEN), dtype=BF16)
        self.status = tw.new_status()

    def logits(self, tokens: torch.Tensor) -> torch.Tensor:
        """fp32 [T, V]. A layer's feedforward output is the next norm's x, the stream its
        residual, so the add and the norm are one pass."""
        stream, out = self.embed.forward(tokens, self.E), None
        self.inputs, self.streams = [], []
        for layer, norm, ffn in zip(self.layers, self.norms, self.ffns):
            h, stream = norm.forward(stream if out is None else out, layer["norm_w"], residual=None if out is None else stream)
            self.inputs.append(h)
            self.streams.append(stream)
            out = ffn.forward(h, layer["Wg"], layer["Wu"], layer["Wd"])
        h, stream = self.norms[-1].forward(out, self.norm_w, residual=stream)
        self.inputs.append(h)
        self.streams.append(stream)
        return tw.dense_gemm(h, self.E, self.T, self.V, self.d, False, False, status=self.status)

    def step(self, tokens: torch.Tensor, labels: torch.Tensor):
        """Losses [T] and the gradients of every weight for the mean loss (plus l1 * the
        activations' sum)."""
        z = self.logits(tokens)
        losses, dz = self.loss.forward_backward(z, labels=labels, scale=1.0 / self.T, out=z)
        dz = dz.to(BF16)
        dh = tw.dense_gemm(dz, self.E, self.T, self.d, self.V, False, True, status=self.status).to(BF16)
        grads = dict(E=tw.dense_gemm(dz, self.inputs[-1], self.V, self.d, self.T, True, True, status=self.status))
        stream_grad, grads["norm_w"] = self.norms[-1].backward(dh, self.streams[-1], self.norm_w)
        grads["layers"] = [None] * len(self.layers)
        for n in reversed(range(len(self.layers))):
            layer = self.layers[n]
            dh, dWg, dWu, dWd = self.ffns[n].backward(stream_grad, self.inputs[n], layer["Wg"], layer["Wu"], layer["Wd"],
                                                      l1=self.l1)
            # what reaches the stream: through the norm, and past the block
            stream_grad, dw = self.norms[n].backward(dh, self.streams[n], layer["norm_w"], dres=stream_grad)
            grads["layers"][n] = dict(norm_w=dw, Wg=dWg, Wu=dWu, Wd=dWd)
        self.embed.backward(stream_grad, tokens, out=grads["E"], add=True)
        return losses, grads

    def update(self, grads, lr: float, hidden_lr: float) -> None:
        """In place: hidden matrices W = (1 - hidden_lr decay) W - hidden_lr sqrt(max(1, I / d))
        times the orthogonalised momentum, the others W - lr gradient."""
        for layer, buffers, g in zip(self.layers, self.momentum, grads["layers"]):
            rows, cols = g["Wg"].shape
            self.ortho([g[k] for k in HIDDEN], [buffers[k] for k in HIDDEN], out=[layer[k] for k in HIDDEN],
                       scale=-hidden_lr * max(1.0, rows / cols) ** 0.5, beta=1.0 - hidden_lr * self.decay)
            layer["norm_w"].sub_(lr * g["norm_w"])
        self.norm_w.sub_(lr * grads["norm_w"])
        self.E.sub_((lr * grads["E"]).to(BF16))

    def check(self) -> None:
        """Raises what the device reported (synchronises)."""
        reported = [("product", self.status), ("loss", self.loss.status), ("embedding", self.embed.status),
                    ("update", self.ortho.status)] + [("ffn", f.status) for f in self.ffns]
        for where, s in reported:
            tw.raise_if_device_error(s, where)


def sequence(T: int, V: int, seed: int = 1):
    """Tokens of a small grammar (a token's successor is one of two) and the next of each; the
    last has none."""
    g = torch.Generator().manual_seed(seed)
    after = torch.randint(0, V, (V, 2), generator=g)
    pick = torch.randint(0, 2, (T,), generator=g).tolist()
    tok = [0]
    for n in range(T - 1):
        tok.append(int(after[tok[-1], pick[n]]))
    tokens = torch.tensor(tok, dtype=torch.int32)
    labels = torch.cat([tokens[1:], torch.tensor([-1], dtype=torch.int32)])
    return tokens.cuda(), labels.cuda()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    T, d, I, V = a.tokens, 512, 1408, 1024
    model = Model(T, d, I, V, layers=2, l1=1e-7)
    tokens, labels = sequence(T, V)
    score = tw.TokenLogprobs(T, V, n_tokens=1, top_k=1, dtype=F32)
    for n in range(a.steps):
        losses, grads = model.step(tokens, labels)
        model.update(grads, lr=0.5, hidden_lr=0.02)
        if n % 5 == 0 or n == a.steps - 1:
            mean = losses.mean().item()
            logprob, entropy, top, _ = score(model.logits(tokens), labels)
            hit = (top[:, 0] == labels)[:-1].float().mean().item()
            print(f"step {n:3d}  loss {mean:.4f}  label log probability {logprob[:-1].mean().item():.3f}  "
                  f"entropy {entropy.mean().item():.3f}  top-1 agreement {hit:.3f}")
    model.check()


if __name__ == "__main__":
    main()
