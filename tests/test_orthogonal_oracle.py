"""Pins of the fp64 oracle of the orthogonal maps, and of the frequencies (CPU)."""
import math

import numpy as np
import pytest

from oracle import orthogonal as oo

QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_product_with_rotation_matrices(interleaved):
    rng = np.random.default_rng(1)
    f = np.array([1.0, 0.1, 0.01])
    x = rng.standard_normal((5, 2, 8))
    p = np.array([0, 1, -3, 7, 1000])
    got = oo.rotary(x, p, f, interleaved, 1.5)
    for t in range(5):
        R = np.eye(8)
        for i in range(3):
            u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
            a = p[t] * f[i]
            R[u, u] = R[v, v] = 1.5 * math.cos(a)
            R[u, v], R[v, u] = -1.5 * math.sin(a), 1.5 * math.sin(a)
        assert np.allclose(got[t], x[t] @ R.T, rtol=1e-12, atol=1e-12)


def test_rotation_keeps_products_of_rows_by_their_distance():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 6)), rng.standard_normal((1, 1, 6))
    f = np.array([0.7, 0.3, 0.01])
    dots = [np.sum(oo.rotary(q, [m + 5], f) * oo.rotary(k, [m], f)) for m in (0, 3, 100, -40)]
    assert np.allclose(dots, dots[0], rtol=1e-12)


def test_gradient_of_rotation_is_its_adjoint():
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 4, 3, 10)), rng.standard_normal((2, 4, 3, 10))
    p, f = rng.integers(-50, 50, (2, 4)), rng.random(4)
    lhs = np.sum(g * oo.rotary(x, p, f, True, 0.7))
    back = oo.rotary(g, p, f, True, 0.7, inverse=True)
    assert np.isclose(lhs, np.sum(back * x), rtol=1e-12)
    step = 1e-6
    for at in [(0, 0, 0, 0), (1, 3, 2, 7), (0, 2, 1, 9)]:
        y = x.copy()
        y[at] += step
        change = (np.sum(g * oo.rotary(y, p, f, True, 0.7)) - lhs) / step
        assert np.isclose(change, back[at], rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (5, 1), (1, 1)])
@pytest.mark.parametrize("steps", [0, 1, 5])
def test_orthogonalisation_is_the_polynomial_of_the_singular_values(shape, steps):
    rng = np.random.default_rng(4)
    g = rng.standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt(np.sum(s * s)) + 1e-7)
    for _ in range(steps):
        s = QUINTIC[0] * s + QUINTIC[1] * s ** 3 + QUINTIC[2] * s ** 5
    assert np.allclose(oo.orthogonalize(g, steps, QUINTIC), (u * s) @ vt, atol=1e-12)


def test_convergent_coefficients_give_the_polar_factor():
    rng = np.random.default_rng(5)
    g = rng.standard_normal((3, 7))
    u, _, vt = np.linalg.svd(g, full_matrices=False)
    assert np.allclose(oo.orthogonalize(g, 12, (15 / 8, -10 / 8, 3 / 8)), u @ vt, atol=1e-9)
    many = np.stack([g, 2.0 * g])
    both = oo.orthogonalize(many, 3, [QUINTIC, QUINTIC, (1.5, -0.5, 0.0)])
    assert np.allclose(both[0], both[1], atol=1e-6)


def test_step_without_momentum_and_decay_is_the_update_alone():
    rng = np.random.default_rng(6)
    w, g = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))
    w2, m2 = oo.step(w, g, np.zeros_like(g), 0.1, 0.0, True, 0.0, 2.0, 5, QUINTIC)
    assert np.allclose(w2, w - 0.2 * oo.orthogonalize(g, 5, QUINTIC)) and np.array_equal(m2, g)


def test_frequencies():
    torch = pytest.importorskip("torch")
    import dense_tensor_decomposition_gb300 as mk
    f = mk.rotary_frequencies(8)
    assert f.dtype == torch.float64 and f.device.type == "cpu"
    assert np.allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(mk.rotary_frequencies(8, scaling="linear", factor=4.0).numpy(), f.numpy() / 4, rtol=1e-14)
    g = mk.rotary_frequencies(8, scaling="base", factor=4.0).numpy()
    assert np.isclose(g[0], 1.0) and np.isclose(g[-1], f[-1] / 4, rtol=1e-12)
    for scaling in ("parts", "turns"):
        h = mk.rotary_frequencies(64, scaling=scaling, factor=8.0, length=4096, low=1.0, high=32.0).numpy()
        plain = mk.rotary_frequencies(64).numpy()
        turns = plain * 4096 / (2 * math.pi)
        assert np.allclose(h[turns > 60], plain[turns > 60], rtol=1e-14)
        assert np.allclose(h[turns < 0.5], plain[turns < 0.5] / 8, rtol=1e-14)
        assert np.all(h <= plain * (1 + 1e-14)) and np.all(h >= plain / 8 * (1 - 1e-14)) and np.all(np.diff(h) < 0)
    h = mk.rotary_frequencies(64, scaling="turns", factor=8.0, length=4096, low=1.0, high=4.0).numpy()
    middle = np.argmin(np.abs(turns - 2.5))
    share = (turns[middle] - 1) / 3
    assert np.isclose(h[middle], plain[middle] * (share + (1 - share) / 8), rtol=1e-12)
    for bad in (dict(dims=7), dict(dims=0), dict(dims=8, base=0.0), dict(dims=8, factor=0.0),
                dict(dims=8, scaling="other"), dict(dims=2, scaling="base"), dict(dims=8, scaling="parts"),
                dict(dims=8, scaling="turns", length=100, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            mk.rotary_frequencies(**bad)
