"""Pins of the fp64 oracle of the sampled operators (CPU): gradients against
differences of the forward formulas and against independent forms of the same sum."""
import numpy as np
import pytest

import oracle
from oracle import sampled as os_


def model(seed, dims, R, S):
    rng = np.random.default_rng(seed)
    A = [rng.standard_normal((n, R)) for n in dims]
    c = np.stack([rng.integers(-1, n + 1, S) for n in dims], axis=1)     # some out of range
    return rng, A, c


def test_lookup_and_gradient_are_adjoint():
    """<g, lookup(T)> = <gradient(g), T> for every g and T."""
    rng = np.random.default_rng(1)
    T = rng.standard_normal((11, 5))
    idx = rng.integers(-2, 13, (7, 9))
    g = rng.standard_normal((7, 9, 5))
    lhs = np.sum(g * os_.embedding(T, idx, 0.3))
    rhs = np.sum(os_.embedding_grad(idx, g, 11, 0.3) * T)
    assert np.isclose(lhs, rhs, rtol=1e-13)


def test_lookup_is_a_product_with_one_hot_rows():
    rng = np.random.default_rng(2)
    T = rng.standard_normal((6, 4))
    idx = np.array([3, -1, 0, 6, 5, 3])
    hot = (idx[:, None] == np.arange(6)).astype(float)
    assert np.allclose(os_.embedding(T, idx, 2.0), 2.0 * hot @ T, rtol=1e-15)
    g = rng.standard_normal((6, 4))
    assert np.allclose(os_.embedding_grad(idx, g, 6, 2.0), 2.0 * hot.T @ g, rtol=1e-14)


@pytest.mark.parametrize("dims,R", [((7,), 3), ((5, 4), 3), ((4, 5, 3), 6), ((3, 2, 4, 3), 2)])
def test_entries_match_the_dense_model(dims, R):
    rng, A, c = model(3 + len(dims), dims, R, 40)
    letters = "abcdef"[:len(dims)]
    dense = np.einsum(",".join(x + "r" for x in letters) + "->" + letters, *A)
    want = [dense[tuple(s)] if all(0 <= i < n for i, n in zip(s, dims)) else 0.0 for s in c]
    assert np.allclose(os_.cp_entries(A, c), want, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("dims,R", [((5, 4), 3), ((4, 5, 3), 6), ((3, 2, 4, 3), 2)])
def test_gradient_is_the_mttkrp_of_the_sampled_tensor(dims, R):
    rng, A, c = model(30 + len(dims), dims, R, 60)
    A = [a.astype(np.float32) for a in A]
    g = rng.standard_normal(60).astype(np.float32)
    Y = np.zeros(dims)
    for s, v in zip(c, g):
        if all(0 <= i < n for i, n in zip(s, dims)):
            Y[tuple(s)] += v
    G = os_.cp_entries_grad(A, c, g)
    for n in range(len(dims)):
        want = oracle.mttkrp(Y.astype(np.float32), A, n)
        assert np.allclose(G[n], want, rtol=1e-5, atol=1e-5)     # Y is rounded to fp32 for the oracle


@pytest.mark.parametrize("dims,R", [((6,), 2), ((4, 5, 3), 3)])
def test_gradient_matches_differences(dims, R):
    rng, A, c = model(50 + len(dims), dims, R, 30)
    g = rng.standard_normal(30)
    G = os_.cp_entries_grad(A, c, g)
    h = 1e-5
    for n, a in enumerate(A):
        for at in np.ndindex(*a.shape):
            up, down = [x.copy() for x in A], [x.copy() for x in A]
            up[n][at] += h
            down[n][at] -= h
            diff = np.sum(g * (os_.cp_entries(up, c) - os_.cp_entries(down, c))) / (2 * h)
            assert abs(diff - G[n][at]) <= 1e-8 * (1 + abs(G[n][at]))


def test_clip_scales_to_the_norm():
    rng = np.random.default_rng(9)
    ts = [rng.standard_normal(s) for s in ((3, 4), (5,), (0,), (2, 2, 2))]
    norm, ys = os_.clip(ts, 0.5, 0.0)
    assert np.isclose(norm, np.linalg.norm(np.concatenate([t.ravel() for t in ts])), rtol=1e-14)
    assert np.isclose(np.linalg.norm(np.concatenate([y.ravel() for y in ys])), 0.5, rtol=1e-14)
    _, same = os_.clip(ts, 100.0)
    assert all(np.array_equal(a, b) for a, b in zip(ts, same))
