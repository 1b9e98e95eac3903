"""fp64 rotations by position, orthogonalisation and its training step (TEST
INFRASTRUCTURE ONLY: only tests/ import it), from the definitions in include/mttkrp.h:

    rotary         (u, v) -> scale (u cos a - v sin a, u sin a + v cos a), a = p f_i, of pair i
    orthogonalize  X = G / (|G|_F + eps), then X <- (a I + b X X^T + c (X X^T)^2) X a step
    step           M' = mu M + G, U = G + mu M' (or M'), W' = (1 - lr wd) W - lr s O(U)

Pins (tests/test_orthogonal_oracle.py): rotations as a product with a rotation matrix, as
what keeps norms and differences of positions; orthogonalisation as the polynomial of the
singular values.
"""
from __future__ import annotations

import numpy as np


def rotary(x, positions, frequencies, interleaved=False, scale=1.0, inverse=False) -> np.ndarray:
    """x: (..., heads, width), positions: what broadcasts to x.shape[:-2]; angles modulo a turn
    by whole positions (exact), in longdouble."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(frequencies, dtype=np.float64)
    p = np.asarray(positions).astype(np.longdouble)
    a = (p[..., None] * f.astype(np.longdouble)).astype(np.longdouble)
    c, s = np.cos(a).astype(np.float64)[..., None, :], np.sin(a).astype(np.float64)[..., None, :]
    if inverse:
        s = -s
    n = len(f)
    out = x.copy()
    iu, iv = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    u, v = x[..., iu], x[..., iv]
    out[..., iu] = scale * (u * c - v * s)
    out[..., iv] = scale * (u * s + v * c)
    return out


def orthogonalize(g, steps, coefficients, eps=1e-7) -> np.ndarray:
    """g: (..., rows, cols); coefficients: a triple, or one for every step."""
    g = np.asarray(g, dtype=np.float64)
    norm = np.sqrt(np.sum(g * g, axis=(-2, -1), keepdims=True))
    x = g / (norm + eps)
    tall = g.shape[-2] > g.shape[-1]
    x = np.swapaxes(x, -1, -2) if tall else x
    table = np.broadcast_to(np.asarray(coefficients, dtype=np.float64), (steps, 3))
    for a, b, c in table:
        gram = x @ np.swapaxes(x, -1, -2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    return np.swapaxes(x, -1, -2) if tall else x


def step(w, g, m, lr, momentum, nesterov, weight_decay, scale, steps, coefficients, eps=1e-7):
    """(W', M')."""
    w, g, m = (np.asarray(t, dtype=np.float64) for t in (w, g, m))
    kept = momentum * m + g
    update = g + momentum * kept if nesterov else kept
    return (1.0 - lr * weight_decay) * w - lr * scale * orthogonalize(update, steps, coefficients, eps), kept
