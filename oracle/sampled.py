"""fp64 lookups, their gradients and clipping (TEST INFRASTRUCTURE ONLY: only
tests/ import it), from the definitions in include/mttkrp.h:

    embedding        out[t] = scale * table[idx_t]
    embedding_grad   out[v] = scale * sum over t with idx_t = v of grad[t]
    cp_entries       x_s = sum_r prod_n A_n(c_sn, r)
    cp_entries_grad  G_n(i) = sum over s with c_sn = i of g_s prod over m != n of A_m(c_sm)
    clip             norm = sqrt(sum x^2), y = x * min(1, max_norm / (norm + eps))

Tokens and samples with an index out of range take no part (a row of zeros, a zero
entry, no contribution to a sum).

Pins (tests/test_sampled_oracle.py): the gradients against differences of the
forward formulas and as their adjoints, the entries against the dense model, their
gradient against the MTTKRP oracle on the tensor that holds g at the coordinates.
"""
from __future__ import annotations

import numpy as np


def embedding(table, idx, scale: float = 1.0) -> np.ndarray:
    table, idx = np.asarray(table, dtype=np.float64), np.asarray(idx)
    out = np.zeros((*idx.shape, table.shape[1]))
    for at in np.ndindex(*idx.shape):
        if 0 <= idx[at] < len(table):
            out[at] = scale * table[idx[at]]
    return out


def embedding_grad(idx, grad, rows: int, scale: float = 1.0) -> np.ndarray:
    idx = np.asarray(idx).reshape(-1)
    grad = np.asarray(grad, dtype=np.float64)
    grad = grad.reshape(len(idx), grad.shape[-1])
    out = np.zeros((rows, grad.shape[-1]))
    inside = (idx >= 0) & (idx < rows)
    np.add.at(out, idx[inside], scale * grad[inside])
    return out


def _inside(factors, coords):
    dims = np.array([len(a) for a in factors])
    return ((coords >= 0) & (coords < dims)).all(axis=1)


def cp_entries(factors, coords) -> np.ndarray:
    factors = [np.asarray(a, dtype=np.float64) for a in factors]
    coords = np.asarray(coords)
    ok = _inside(factors, coords)
    x = np.zeros(len(coords))
    x[ok] = np.prod([a[coords[ok, n]] for n, a in enumerate(factors)], axis=0).sum(axis=1)
    return x


def cp_entries_grad(factors, coords, g) -> list[np.ndarray]:
    factors = [np.asarray(a, dtype=np.float64) for a in factors]
    coords = np.asarray(coords)
    ok = _inside(factors, coords)
    coords, g = coords[ok], np.asarray(g, dtype=np.float64)[ok]
    rows = [a[coords[:, n]] for n, a in enumerate(factors)]
    out = []
    for n, a in enumerate(factors):
        term = np.repeat(g[:, None], a.shape[1], axis=1)
        for m in range(len(factors)):
            if m != n:
                term = term * rows[m]
        G = np.zeros_like(a)
        np.add.at(G, coords[:, n], term)
        out.append(G)
    return out


def clip(tensors, max_norm: float, eps: float = 1e-6):
    """(norm, clipped tensors)"""
    tensors = [np.asarray(t, dtype=np.float64) for t in tensors]
    norm = np.sqrt(sum(float(np.sum(t * t)) for t in tensors))
    coef = min(1.0, max_norm / (norm + eps))
    return norm, [coef * t for t in tensors]
