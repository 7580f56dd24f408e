"""Orthogonalised updates in float64: momentum and Newton-Schulz steps as defined, on the
matrix as given (no transposing, no scaling by powers of two, no other form of the step)."""
from __future__ import annotations

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def momentum(g, buf, mu, nesterov=True):
    """(new buffer, update)."""
    new = mu * buf + g
    return new, (g + mu * new if nesterov else new)


def newton_schulz(u, steps=5, coefficients=COEFFICIENTS):
    """X after `steps` of X <- a X + (b A + c A^2) X, A = X X^T, from u / |u|_F. coefficients:
    one triple, or one for each step."""
    rows = [coefficients] * steps if np.ndim(coefficients) == 1 else list(coefficients)
    norm = np.sqrt((u * u).sum())
    x = u / norm if norm > 0 else np.zeros_like(u)
    for a, b, c in rows:
        if x.shape[0] <= x.shape[1]:
            gram = x @ x.T
            x = a * x + (b * gram + c * gram @ gram) @ x
        else:  # the same product, taken from the right: A X = X (X^T X)
            gram = x.T @ x
            x = a * x + x @ (b * gram + c * gram @ gram)
    return x
