"""Definitions in float64 of the operators at the ends of a model around the
feedforward layer: layer norm, distillation from a teacher's top logits, and token log
probabilities. Plain numpy; infinities follow the conventions of include/twell.h."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------- layer norm

def layer_norm(s, weight=None, bias=None, eps=1e-5):
    """y, mean, rstd of the rows of s (the residual stream, already added)."""
    s = np.asarray(s, dtype=np.float64)
    mean = s.mean(axis=1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (s - mean[:, None]) * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_grad(dy, s, weight=None, eps=1e-5, dres=None):
    """dx, dweight, dbias of sum(dy * y) (+ sum(dres * s))."""
    dy = np.asarray(dy, dtype=np.float64)
    xh, _, rstd = layer_norm(s, eps=eps)
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xh * (g * xh).mean(axis=1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ---------------------------------------------------------------------- distillation

def _lse(v):
    m = np.max(v) if v.size else -np.inf
    return m if np.isinf(m) else m + np.log(np.exp(v - m).sum())


def _distill_row(z, idx, val, rest, label, tau, kd_w, ce_w):
    """loss and dz of one row (upstream gradient 1)."""
    V = z.size
    entries = [(int(i), float(v) / tau) for i, v in zip(idx, val) if i >= 0]
    buckets = np.array([t for _, t in entries] + [rest])
    lse_t = _lse(buckets)
    some, has = kd_w != 0 and lse_t != -np.inf, ce_w != 0 and label >= 0
    dz = np.zeros(V)
    if not some and not has:
        return 0.0, dz
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.nan, np.full(V, np.nan)
    if np.isneginf(z).all():
        return np.inf, dz
    loss = 0.0
    if some:
        P = np.exp(buckets - lse_t)
        logP = buckets - lse_t
        logq = z / tau - _lse(z / tau)
        listed = np.zeros(V, dtype=bool)
        listed[[i for i, _ in entries]] = True
        log_rest = _lse(logq[~listed])
        kd = sum(P[k] * (logP[k] - logq[i]) for k, (i, _) in enumerate(entries) if P[k] > 0)
        if P[-1] > 0:
            kd += P[-1] * (logP[-1] - log_rest)
        pt = np.zeros(V)
        for k, (i, _) in enumerate(entries):
            pt[i] += P[k]
        if P[-1] > 0 and log_rest > -np.inf:
            zr = z[~listed] / tau  # q / q_rest: log q - log q_rest would lose the count of tokens at -3e38
            e = np.exp(zr - zr.max())
            pt[~listed] += P[-1] * e / e.sum()
        loss += kd_w * tau * tau * kd
        dz += kd_w * tau * (np.exp(logq) - pt)
    if has:
        logp = z - _lse(z)
        loss -= ce_w * logp[label]
        dz += ce_w * np.exp(logp)
        dz[label] -= ce_w
    return loss, dz


def distill(z, idx=None, val=None, rest=None, labels=None, temperature=1.0, kd_weight=1.0, ce_weight=0.0, dloss=None,
            scale=1.0):
    """losses [N], dz [N, V]."""
    z = np.asarray(z, dtype=np.float64)
    N = z.shape[0]
    loss, dz = np.zeros(N), np.zeros(z.shape)
    with np.errstate(invalid="ignore", divide="ignore"):
        for n in range(N):
            loss[n], dz[n] = _distill_row(z[n], [] if idx is None else idx[n], [] if idx is None else val[n],
                                          -np.inf if rest is None else float(rest[n]),
                                          -1 if labels is None else int(labels[n]), temperature, kd_weight, ce_weight)
            dz[n] *= scale * (1.0 if dloss is None else float(dloss[n]))
    return loss, dz


# ---------------------------------------------------------------------- token log probabilities

def token_logprobs(z, tokens, top_k=0, temperature=1.0):
    """logprob [N, S], entropy [N], top_idx [N, top_k], top_logprob [N, top_k]."""
    z = np.asarray(z, dtype=np.float64)
    N, V = z.shape
    logprob = np.zeros(tokens.shape)
    entropy = np.zeros(N)
    top_idx = np.full((N, top_k), -1, dtype=np.int32)
    top_lp = np.full((N, top_k), -np.inf)
    for n in range(N):
        if np.isnan(z[n]).any() or np.isposinf(z[n]).any():
            lp = np.full(V, np.nan)
            entropy[n], top_lp[n] = np.nan, np.nan
        elif np.isneginf(z[n]).all():
            lp = np.full(V, -np.inf)
        else:
            lp = z[n] / temperature - _lse(z[n] / temperature)
            p = np.exp(lp)
            entropy[n] = -(p[p > 0] * lp[p > 0]).sum()
            order = np.argsort(-(z[n] + 0.0), kind="stable")
            order = order[~np.isneginf(z[n][order])][:top_k]
            top_idx[n, :order.size] = order
            top_lp[n, :order.size] = lp[order]
        for s, t in enumerate(tokens[n]):
            logprob[n, s] = 0.0 if t < 0 else lp[t]
    return logprob, entropy, top_idx, top_lp
