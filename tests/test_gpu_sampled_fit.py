"""The example that runs the sampled operators together: one step against the fp64
oracle, the objective's differences along its gradient, and a fit that converges."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import sampled as os_

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sampled_cp_fit.py")
    spec = importlib.util.spec_from_file_location("sampled_cp_fit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def objective(A, c, y, penalty):
    rows = sum(np.sum(a[c[:, n]] ** 2) for n, a in enumerate(A))
    return np.mean((os_.cp_entries(A, c) - y) ** 2) + penalty * rows / len(c)


@pytest.mark.parametrize("dims,R,S,max_norm", [((30, 20, 25), 6, 2000, None), ((30, 20, 25), 6, 2000, 0.05),
                                               ((9, 400), 33, 30000, 0.01)])
def test_a_step_is_the_objectives_gradient(dims, R, S, max_norm):
    ex = example()
    coords, values = ex.samples(dims, 3, S)
    gen = torch.Generator(device="cuda").manual_seed(5)
    A = [torch.randn(n, R, generator=gen, device="cuda") * 0.4 for n in dims]
    loss, grads, norm = ex.gradients(A, coords, values, 0.01, max_norm)
    A64, c, y = [a.double().cpu().numpy() for a in A], coords.cpu().numpy(), values.double().cpu().numpy()
    x = os_.cp_entries(A64, c)
    G = os_.cp_entries_grad(A64, c, 2.0 / S * (x - y))
    G = [g + os_.embedding_grad(c[:, n], 2.0 * 0.01 / S * A64[n][c[:, n]], dims[n]) for n, g in enumerate(G)]
    want_norm, clipped = os_.clip(G, 1e30 if max_norm is None else max_norm)
    assert abs(float(loss) - np.mean((x - y) ** 2)) <= 1e-5 * np.mean((x - y) ** 2)
    # the residual carries the entries' rounding: relative to the terms' magnitudes, (R + 4) u,
    # next to the sums' own (S + 4) u
    mag = os_.cp_entries_grad([np.abs(a) for a in A64], c, 2.0 / S * (os_.cp_entries([np.abs(a) for a in A64], c) + np.abs(y)))
    mag = [m + os_.embedding_grad(c[:, n], 2.0 * 0.01 / S * np.abs(A64[n][c[:, n]]), dims[n]) for n, m in enumerate(mag)]
    scale = 1.0 if max_norm is None else min(1.0, max_norm / want_norm)
    for n, g in enumerate(grads):
        count = np.bincount(c[:, n], minlength=dims[n])[:, None]
        assert np.all(np.abs(g.double().cpu().numpy() - clipped[n]) <= (2 * count + R + 40) * U * mag[n] * scale)
    assert abs(float(norm) - want_norm) <= 1e-5 * want_norm
    if max_norm is None:
        h = 1e-6
        for n in range(len(dims)):
            D = np.random.default_rng(n).standard_normal(A64[n].shape)
            up, down = [a.copy() for a in A64], [a.copy() for a in A64]
            up[n] += h * D
            down[n] -= h * D
            diff = (objective(up, c, y, 0.01) - objective(down, c, y, 0.01)) / (2 * h)
            assert abs(diff - np.sum(G[n] * D)) <= 1e-6 * np.sum(np.abs(G[n] * D))


def test_the_fit_converges():
    ex = example()
    dims = (40, 30, 20)
    coords, values = ex.samples(dims, 3, 20000)
    factors, losses = ex.fit(coords, values, dims, 6, 300, 4096)
    losses = losses.cpu().numpy()
    assert np.isfinite(losses).all() and losses[:5].mean() > 0.5 and losses[-20:].mean() < 0.05
    again, _ = ex.fit(coords, values, dims, 6, 300, 4096)
    assert all(torch.equal(a, b) for a, b in zip(factors, again))      # the whole fit repeats bit by bit
