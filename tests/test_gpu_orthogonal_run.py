"""The orthogonal maps where they are used: one training step of a table whose rows are turned by
their position (lookup, rotation, loss, rotation back, gradient of the table, clipping, update by
orthogonalised momentum) against the fp64 oracles and differences, and the fit of the example."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import orthogonal as oo
from oracle import sampled as os_

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sampled_cp_fit.py")
    spec = importlib.util.spec_from_file_location("sampled_cp_fit", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def loss64(table, idx, at, f, w, y):
    """mean over tokens of (<rotated row, w> - y)^2"""
    z = oo.rotary(os_.embedding(table, idx)[:, None], at, f)[:, 0]
    return np.mean((z @ w - y) ** 2)


def one_step(table, momentum, idx, at, f, w, y, outs):
    rows = mk.embedding(table, idx)
    z = mk.rotary(rows, at, f)
    residual = z @ w - y
    dz = (2.0 / len(idx)) * residual[:, None] * w
    drows = mk.rotary_grad(dz, at, f)
    grad = mk.embedding_grad(idx, drows, table.shape[0])
    norm = mk.clip_grad_norm([grad], 0.05)
    mk.orthogonal_step([table], [grad], [momentum], 0.01, momentum=0.9, weight_decay=0.1, outs=outs[:1], momenta_outs=outs[1:])
    return residual.square().mean(), grad, norm


@pytest.mark.parametrize("V,D,T", [(50, 24, 700), (400, 160, 3000)])
def test_a_training_step_of_rows_with_positions(V, D, T):
    gen = torch.Generator(device="cuda").manual_seed(V)
    table = torch.randn(V, D, generator=gen, device="cuda") * 0.3
    momentum = torch.randn(V, D, generator=gen, device="cuda") * 1e-3
    idx = torch.randint(0, V, (T,), generator=gen, device="cuda")
    at = torch.randint(0, 100000, (T,), generator=gen, device="cuda")
    w, y = torch.randn(D, generator=gen, device="cuda"), torch.randn(T, generator=gen, device="cuda")
    f = mk.rotary_frequencies(D)
    outs = [torch.empty_like(table), torch.empty_like(table)]
    torch.backends.cuda.matmul.allow_tf32 = False
    loss, grad, norm = one_step(table, momentum, idx, at, f, w, y, outs)
    n64 = lambda t: t.double().cpu().numpy()
    A, i, p, w64, y64, f64 = n64(table), idx.cpu().numpy(), at.cpu().numpy(), n64(w), n64(y), f.numpy()
    z = oo.rotary(A[i][:, None], p, f64)[:, 0]
    residual = z @ w64 - y64
    G = os_.embedding_grad(i, oo.rotary((2.0 / T * residual[:, None] * w64)[:, None], p, f64, inverse=True)[:, 0], V)
    assert abs(float(loss) - np.mean(residual ** 2)) <= 1e-5 * np.mean(residual ** 2)
    # the residual is a sum of D products of rotated rows (each within 8 u, twice for the pair)
    # in any order, and of y; the gradient's terms are rotated once more, and a sum of those of a row
    size = np.abs(A[i]).sum(1) * np.abs(w64).max() * 2 + np.abs(y64)
    terms = 2.0 / T * ((D + 20) * U * size)[:, None] * np.abs(w64).max() * 2 * np.ones((1, D))
    count = np.bincount(i, minlength=V)[:, None]
    mag = os_.embedding_grad(i, 2.0 / T * np.abs(residual)[:, None] * np.abs(w64).max() * 2 * np.ones((1, D)), V)
    bound = os_.embedding_grad(i, terms, V) + (count + 20) * U * mag
    want_norm, (clipped,) = os_.clip([G], 0.05)
    share = min(1.0, 0.05 / want_norm)
    assert np.all(np.abs(n64(grad) - clipped) <= bound * share * 1.01 + 1e-5 * np.abs(clipped))
    assert abs(float(norm) - want_norm) <= 1e-5 * want_norm
    # the formula's gradient against differences of the loss
    for seed in range(3):
        d = np.random.default_rng(seed).standard_normal(A.shape)
        h = 1e-6
        diff = (loss64(A + h * d, i, p, f64, w64, y64) - loss64(A - h * d, i, p, f64, w64, y64)) / (2 * h)
        assert abs(diff - np.sum(G * d)) <= 1e-6 * np.sum(np.abs(G * d))
    # the step, from the gradient that the step got
    by = max(1.0, V / D) ** 0.5
    want, want_m = oo.step(A, n64(grad), n64(momentum), 0.01, 0.9, True, 0.1, by, 5, mk.QUINTIC)
    o = oo.orthogonalize(n64(grad) + 0.9 * want_m, 5, mk.QUINTIC)
    assert np.linalg.norm(n64(outs[0]) - want) <= 0.01 * by * 1e-4 * np.linalg.norm(o) + 4 * U * np.linalg.norm(A)
    assert np.abs(n64(outs[1]) - want_m).max() <= 4 * U * np.abs(want_m).max()
    again = [torch.empty_like(table), torch.empty_like(table)]
    one_step(table, momentum, idx, at, f, w, y, again)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


def test_the_example_with_orthogonalised_updates_repeats():
    ex = example()
    dims = (40, 30, 20)
    coords, values = ex.samples(dims, 3, 20000)
    factors, losses = ex.fit(coords, values, dims, 6, 50, 4096, rate=0.02, orthogonal=True)
    assert torch.isfinite(losses).all()
    again, _ = ex.fit(coords, values, dims, 6, 50, 4096, rate=0.02, orthogonal=True)
    assert all(torch.equal(a, b) for a, b in zip(factors, again))
    # its first step, from the gradients of the same batch
    gen = torch.Generator(device="cuda").manual_seed(0)
    start = [torch.randn(n, 6, generator=gen, device="cuda").mul_(0.3) for n in dims]
    pick = torch.randint(coords.shape[0], (4096,), generator=gen, device="cuda")
    _, grads, _ = ex.gradients(start, coords[pick], values[pick], 1e-4, 1.0)
    one, _ = ex.fit(coords, values, dims, 6, 1, 4096, rate=0.02, orthogonal=True)
    for a, g, b in zip(start, grads, one):
        want, _ = oo.step(a.double().cpu(), g.double().cpu(), np.zeros(g.shape), 0.02, 0.9, True, 0.0, 1.0, 5, mk.QUINTIC)
        assert np.linalg.norm(b.double().cpu().numpy() - want) <= 0.02 * 1e-4 * 6 ** 0.5 + 4 * U * np.linalg.norm(want)


def test_two_graphs_at_once():
    """Two captured graphs of all operators, replayed beside one another and beside eager calls, with results of
    their own: workspaces are not shared."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    f = mk.rotary_frequencies(16)
    shapes = [(300, 200), (64, 40), (100, 500), (257, 1033)]
    sets = []
    for _ in range(3):
        x = torch.randn(2, 50, 3, 17, generator=gen, device="cuda")
        p = torch.randint(0, 1000, (2, 50), generator=gen, device="cuda")
        gs = [torch.randn(s, generator=gen, device="cuda") for s in shapes]
        sets.append((x, p, gs))

    def run(x, p, gs):
        return [mk.rotary(x, p, f, True)] + mk.orthogonalize(gs) + mk.orthogonalize(gs, dtype=torch.bfloat16)

    want = [run(*s) for s in sets]
    graphs, got = [], []
    for s in sets[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    eager = []
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager.append(run(*sets[2]))
    torch.cuda.synchronize()
    for a, b in zip(got + eager, want[:2] + 5 * [want[2]]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
