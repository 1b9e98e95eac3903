"""GPU orthogonalisation by Newton-Schulz products and its training step against the fp64 oracle.

Whole numbers.  G of 4^q entries +-1 has the norm 2^q, so X = G / 2^q, and S, S S, P and P X are
whole numbers over powers of two.  While these numbers stay below 2^22 (2^11 where only leading
parts are used) every product and sum here is exact, and results are compared bit by bit, after
one rounding to their type.  This is where tiles, edges, orders and lists are checked.

Coefficients as in use.  An error E of X (Frobenius norm) grows by at most L a step: the largest
divided difference of the odd polynomial p on [-u, u], u the largest singular value reached: |p'| on
[0, u], at most 4.25 for the quintic up to 1.21.  A step's own error: products of two fp16 parts
are within 2^-22 of their terms and of tensor-memory sums that are cut off 24 times between
drains, each by at most 2^-23, and by half of that on average: eta = 2^-20 of |A|_2 |B|_F.  With
|b| u^2 + 3 |c| u^4 for the errors of S and S S, and the bracket's 3.4445, a step adds at most 24 eta
|X|_F.  The bound is the sum over the steps, from the oracle's own |X|_F, plus the rounding of the
result.  For bf16 results eta is 2^-11 (leading parts of S and P)."""
import numpy as np
import pytest

from oracle import orthogonal as oo

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.double().cpu().numpy()


def signs(seed, shape, q):
    """4^q entries +-1 in every matrix, the others 0."""
    rng = np.random.default_rng(seed)
    g = np.zeros(shape)
    for m in g.reshape(-1, shape[-2] * shape[-1]):
        at = rng.choice(m.size, 4 ** q, replace=False)
        m[at] = rng.choice([-1.0, 1.0], 4 ** q)
    return g


def cuda(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


SIZES = [  # rows, cols, q
    (1, 1, 0), (1, 7, 1), (7, 1, 1), (2, 3, 1), (20, 128, 3), (64, 64, 3), (63, 65, 4), (65, 63, 4), (128, 128, 4),
    (130, 129, 4), (129, 400, 5), (400, 129, 5), (256, 64, 4), (300, 300, 5), (513, 257, 5), (257, 513, 5),
    (640, 1000, 6), (1000, 640, 6), (70, 2900, 6), (2900, 70, 6)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("abc", [(1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0), (0.5, -1.0, 0.25)])
@pytest.mark.parametrize("rows,cols,q", SIZES)
def test_one_step_of_whole_numbers(rows, cols, q, abc, dtype):
    g = signs(rows + cols, (rows, cols), q)
    out = mk.orthogonalize(cuda(g), 1, abc, eps=0.0, dtype=TYPES[dtype])
    want = oo.orthogonalize(g, 1, abc, 0.0)
    if abc[0] * abc[2] != 0.0:
        # P has 2 + 4 q bits: the parts' 22 (11 for bf16) do not hold them all for larger ones; what is
        # left out is below 2^-22 (2^-11) of P's entries, which are below 3
        left = 2.0 ** (-11 if dtype == "bfloat16" else -22) * 3
        err = np.abs(f64(out) - want)
        x = np.abs(g) / 2.0 ** q
        assert np.all(err <= left * x.sum(0)[None, :] + left * x.sum(1)[:, None] + UNIT[TYPES[dtype]] * 1.01 * np.abs(want))
        return
    n = g @ g.T if rows <= cols else g.T @ g
    p = n if abc[1] else n @ n if abc[2] else np.eye(len(n))
    if dtype == "bfloat16" and np.abs(p).max() > 2 ** 11:
        # 70 x 2900 with 4096 entries: the diagonal of S S is (4096 / 70)^2 = 3424 and more, above the
        # 11 bits of P's leading part, which is within half a step, 2^-11 of its entry
        p, x = np.abs(p) / 16.0 ** q, np.abs(g) / 2.0 ** q
        left = 2.0 ** -11 * (p @ x if rows <= cols else x @ p)
        assert np.all(np.abs(f64(out) - want) <= left + 2.0 ** -8 * 1.01 * np.abs(want))
    else:
        assert torch.equal(out, cuda(want).to(TYPES[dtype]))


@pytest.mark.parametrize("dtype", TYPES)
def test_two_steps_of_whole_numbers(dtype):
    """The second step reads what the first wrote: X S, then S of that."""
    for rows, cols in ((30, 40), (40, 30), (200, 150), (150, 200)):
        g = signs(rows, (rows, cols), 2)
        out = mk.orthogonalize(cuda(g, TYPES[dtype]), 2, [(0.0, 1.0, 0.0), (0.0, 4.0, 0.0)], eps=0.0)
        want = oo.orthogonalize(g, 2, [(0.0, 1.0, 0.0), (0.0, 4.0, 0.0)], 0.0)
        assert torch.equal(out, cuda(want).to(TYPES[dtype])), (rows, cols)


CLUSTERS = [  # short side, long side, q: a CTA, clusters of 2, 4 and 8 of either kind of kernel, and beyond
    (64, 512, 5), (64, 513, 5), (33, 1000, 5), (1, 2500, 5), (64, 5000, 6), (17, 5120, 6), (17, 5121, 6), (65, 65, 4),
    (128, 192, 5), (100, 193, 5), (128, 500, 5), (65, 1000, 5), (127, 1536, 6), (127, 1537, 6)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("short,long,q", CLUSTERS)
def test_short_sides(short, long, q, tall, dtype):
    """S X, and S of that, in whole numbers; the same for every matrix of a list and a batch."""
    g = signs(short + long, (3, long, short) if tall else (3, short, long), q)
    out = mk.orthogonalize(cuda(g), 1, (0.0, 1.0, 0.0), eps=0.0, dtype=TYPES[dtype])
    want = cuda(oo.orthogonalize(g, 1, (0.0, 1.0, 0.0), 0.0)).to(TYPES[dtype])
    assert torch.equal(out, want)
    each = [cuda(m) for m in g]
    for got, one in zip(mk.orthogonalize(each, 1, (0.0, 1.0, 0.0), eps=0.0, dtype=TYPES[dtype]), want):
        assert torch.equal(got, one)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("abc", [(1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0)])
@pytest.mark.parametrize("count,rows,cols", [(24, 1024, 768), (24, 600, 1100), (24, 1100, 600), (2, 4096, 4033), (5, 3971, 2050)])
def test_pairs_of_ctas(count, rows, cols, abc, dtype):
    """Sizes from which pairs take some or all of the products, in whole numbers: one to three entries
    a row of the smaller side, so that all are small."""
    gen = generator(rows)
    g = torch.zeros(count, rows, cols, device="cuda", dtype=torch.float64)
    at = torch.stack([torch.randperm(rows * cols, generator=gen, device="cuda")[:1024] for _ in range(count)])
    sign = torch.randint(0, 2, at.shape, generator=gen, device="cuda").double() * 2 - 1
    g.view(count, -1).scatter_(1, at, sign)
    out = mk.orthogonalize(g.to(torch.float32), 1, abc, eps=0.0, dtype=TYPES[dtype])
    x = g / 32.0
    x = x.mT if rows > cols else x
    s = x @ x.mT
    want = abc[0] * x + (abc[1] * s + abc[2] * (s @ s)) @ x
    want = want.mT if rows > cols else want
    assert torch.equal(out, want.to(TYPES[dtype]))


def test_long_lists_of_small_matrices():
    """More elements than a launch takes, of both kinds of kernel and several clusters, and large ones between."""
    gen = generator(11)
    shapes = [(8, 8), (20, 128), (128, 20), (64, 700), (100, 100), (128, 400), (300, 200), (1, 1), (70, 900)] * 20
    gs = [gradient(gen, s) for s in shapes]
    got = mk.orthogonalize(gs)
    for s, g, x in zip(shapes, gs, got):
        want = mk.orthogonalize(g)
        # a cluster's size follows the number of matrices: sums are added in another order
        assert float((x - want).norm()) <= 1e-5 * float(want.norm()), s
    assert all(torch.equal(a, b) for a, b in zip(got, mk.orthogonalize(gs)))


def trajectory_bound(g, steps, coefficients, eta):
    """Bound of the error's Frobenius norm, and the oracle's result."""
    total, before = 0.0, oo.orthogonalize(g, 0, coefficients)
    for k in range(steps):
        total = 4.25 * total + 24 * eta * np.linalg.norm(before)
        before = _step(before, coefficients)
    return total, before


def _step(x, abc):
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    s = x @ x.T
    x = abc[0] * x + (abc[1] * s + abc[2] * s @ s) @ x
    return x.T if tall else x


def gradient(gen, shape, dtype=torch.float32, noise=0.1):
    """A few strong directions over noise."""
    r, c = shape
    rank = max(1, min(r, c) // 16)
    u = torch.randn(r, rank, generator=gen, device="cuda")
    v = torch.randn(rank, c, generator=gen, device="cuda")
    return (u @ v / rank ** 0.5 + noise * torch.randn(r, c, generator=gen, device="cuda")).to(dtype)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


SHAPES = [(1, 1), (1, 50), (50, 1), (8, 8), (20, 128), (256, 64), (64, 300), (333, 501), (501, 333), (512, 2000),
          (1100, 900)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_quintic(shape, dtype):
    g = gradient(generator(shape[0]), shape, TYPES[dtype])
    out = mk.orthogonalize(g, scale=0.5)
    assert out.shape == g.shape and out.dtype == g.dtype
    eta = 2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -20
    bound, want = trajectory_bound(f64(g), 5, mk.QUINTIC, eta)
    err = np.linalg.norm(f64(out) - 0.5 * want)
    assert err <= 0.5 * (bound + UNIT[g.dtype] * np.linalg.norm(want)), err / bound
    assert torch.equal(out, mk.orthogonalize(g, scale=0.5))


@pytest.mark.parametrize("noise", [1.0, 1e-1, 1e-2, 1e-4])
def test_as_near_as_fp32(noise):
    """Weak directions are raised by up to 485: results in fp32 are no farther from the 64-bit
    value than twice what the formula in fp32 products gives (or 1e-6), those in bf16 within 2.5e-3:
    1.5e-3 of the products and 2^-9 / sqrt(3) x 1.5 of the rounding, squares added."""
    for shape in ((512, 512), (256, 1024), (1024, 256)):
        g = gradient(generator(7), shape, noise=noise)
        want = oo.orthogonalize(f64(g), 5, mk.QUINTIC)
        x = g / (g.norm() + 1e-7)
        x = x.mT if shape[0] > shape[1] else x
        for _ in range(5):
            s = x @ x.mT
            x = mk.QUINTIC[0] * x + (mk.QUINTIC[1] * s + mk.QUINTIC[2] * (s @ s)) @ x
        x = x.mT if shape[0] > shape[1] else x
        size = np.linalg.norm(want)
        plain = np.linalg.norm(f64(x) - want) / size
        here = np.linalg.norm(f64(mk.orthogonalize(g)) - want) / size
        assert here <= max(2 * plain, 1e-6), (shape, here, plain)
        short = np.linalg.norm(f64(mk.orthogonalize(g, dtype=torch.bfloat16)) - want) / size
        assert short <= 2.5e-3, (shape, short)


def test_convergent_coefficients_make_it_orthogonal():
    g = gradient(generator(1), (300, 120), noise=1.0)
    x = mk.orthogonalize(g, steps=20, coefficients=(15 / 8, -10 / 8, 3 / 8))
    eye = x.double().mT @ x.double()
    # at the fixed point p' = 0: an error is that of the last step alone, 24 eta |X|_F, twice in X^T X
    assert float((eye - torch.eye(120, device="cuda")).norm()) <= 2 * 24 * 2.0 ** -20 * 120 ** 0.5
    u, _, vt = np.linalg.svd(f64(g), full_matrices=False)
    assert np.linalg.norm(f64(x) - u @ vt) <= 24 * 2.0 ** -20 * 120 ** 0.5 * 2


def test_lists_batches_and_strides():
    """Every matrix as if it were alone: lists of mixed shapes and types, batches, parts of wider
    rows, columns for rows, rows at odd offsets, in place."""
    gen = generator(2)
    shapes = [(40, 30), (200, 300), (1, 9), (129, 65), (64, 64), (300, 20)] * 7         # two groups of launches
    types = [torch.float32, torch.bfloat16, torch.float16]
    gs = [gradient(gen, s, types[k % 3]) for k, s in enumerate(shapes)]
    alone = [mk.orthogonalize(g.float(), dtype=torch.float32) for g in gs]
    for got, want in zip(mk.orthogonalize(gs, dtype=torch.float32), alone):
        assert torch.equal(got, want)
    scales = [0.1 * k for k in range(len(gs))]
    for got, want, by in zip(mk.orthogonalize(gs, scale=scales, dtype=torch.float32), alone, scales):
        assert torch.allclose(got, want * by, rtol=2.0 ** -23, atol=0)
    batch = torch.stack([gradient(gen, (70, 90)) for _ in range(12)])
    each = torch.stack([mk.orthogonalize(m) for m in batch])
    assert torch.equal(mk.orthogonalize(batch), each)
    assert torch.equal(mk.orthogonalize(batch.view(3, 4, 70, 90)), each.view(3, 4, 70, 90))
    assert torch.equal(mk.orthogonalize(batch[::2]), each[::2])
    assert torch.equal(mk.orthogonalize(batch.mT), each.mT)
    assert mk.orthogonalize(batch.mT).stride() == batch.mT.stride()
    room = torch.zeros(70, 95, device="cuda")
    for at in (0, 1, 4, 5):
        part = room[:, at:at + 90]
        part.copy_(batch[3])
        assert torch.equal(mk.orthogonalize(part), each[3])
        version = part._version
        assert mk.orthogonalize(part, outs=part).data_ptr() == part.data_ptr() and part._version > version
        assert torch.equal(part, each[3])
        assert room[:, :at].abs().sum() == 0 and room[:, at + 90:].abs().sum() == 0
        room.zero_()
    half = torch.zeros(70, 95, device="cuda", dtype=torch.float16)
    assert torch.equal(mk.orthogonalize(batch[3], outs=half[:, 1:91]), each[3].half())
    # halves of one buffer, side by side and interleaved by rows
    wide = torch.zeros(70, 180, device="cuda")
    a, b = wide[:, :90], wide[:, 90:]
    a.copy_(batch[0])
    b.copy_(batch[1])
    mk.orthogonalize([a, b], outs=[a, b])
    assert torch.equal(a, each[0]) and torch.equal(b, each[1])
    # nothing to do
    assert mk.orthogonalize(batch[:0]).shape == (0, 70, 90)
    got = mk.orthogonalize([batch[0, :0], batch[0], batch[0, :, :0]])
    assert got[0].numel() == 0 and got[2].numel() == 0 and torch.equal(got[1], each[0])


def test_extreme_values():
    gen = generator(3)
    g = gradient(gen, (90, 70))
    base = mk.orthogonalize(g, eps=0.0)
    for by in (2.0 ** 100, 2.0 ** -60, 2.0 ** 110, 2.0 ** -110):      # whatever its size
        got = mk.orthogonalize(g * by, eps=0.0)
        assert float((got - base).norm()) <= 1e-4 * float(base.norm())
    assert mk.orthogonalize(torch.zeros(65, 30, device="cuda")).abs().sum() == 0
    for bad in (float("nan"), float("inf")):
        h = g.clone()
        h[3, 5] = bad
        got = mk.orthogonalize([h, g], eps=0.0)
        assert torch.isnan(got[0]).all() and torch.equal(got[1], base)


MOMENTA = [("float32", "float32", "float32"), ("bfloat16", "bfloat16", "bfloat16"), ("float32", "bfloat16", "float32"),
           ("float16", "float32", "bfloat16")]


@pytest.mark.parametrize("weights,grads,momenta", MOMENTA)
@pytest.mark.parametrize("nesterov", [False, True])
def test_step(weights, grads, momenta, nesterov):
    gen = generator(4)
    shapes = [(90, 70), (70, 301), (257, 128), (2, 33, 47)]

    def make(s, dtype, by):
        if len(s) == 3:
            return torch.stack([gradient(gen, s[1:]) for _ in range(s[0])]).mul(by).to(dtype)
        return gradient(gen, s).mul(by).to(dtype)

    g = [make(s, TYPES[grads], 1e-3) for s in shapes]
    m = [make(s, TYPES[momenta], 5e-3) for s in shapes]
    w = [torch.randn(s, generator=gen, device="cuda").mul(0.02).to(TYPES[weights]) for s in shapes]
    outs, kept = [torch.zeros_like(x) for x in w], [torch.zeros_like(x) for x in m]
    before = [x.clone() for x in w + m + g]
    got = mk.orthogonal_step(w, g, m, 0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, outs=outs, momenta_outs=kept)
    assert [x.data_ptr() for x in got] == [x.data_ptr() for x in outs]
    assert all(torch.equal(x, y) for x, y in zip(w + m + g, before))
    eta = 2.0 ** -11 if weights == "bfloat16" else 2.0 ** -20
    for k, s in enumerate(shapes):
        by = max(1.0, s[-2] / s[-1]) ** 0.5
        want, want_m = oo.step(f64(w[k]), f64(g[k]), f64(m[k]), 0.02, 0.9, nesterov, 0.1, by, 5, mk.QUINTIC)
        # one fused product and sum: 2 roundings of fp32, then the type's
        size = 0.9 * np.abs(f64(m[k])) + np.abs(f64(g[k]))
        assert np.all(np.abs(f64(kept[k]) - want_m) <= 2.0 ** -23 * size + UNIT[m[k].dtype] * 1.01 * np.abs(want_m) + 2.0 ** -25)
        for i in np.ndindex(s[:-2]):
            u = 0.9 * f64(m[k])[i] + f64(g[k])[i]
            u = f64(g[k])[i] + 0.9 * u if nesterov else u
            bound, o = trajectory_bound(u, 5, mk.QUINTIC, eta)
            # rounding to fp32 of U (a 2^-23 error of X, grown by L^5) and of W's formula
            bound += 4.25 ** 5 * 2.0 ** -23
            size = np.linalg.norm(f64(w[k])[i]) + 0.02 * by * np.linalg.norm(o)
            err = np.linalg.norm(f64(outs[k])[i] - want[i])
            assert err <= 0.02 * by * bound + 2.0 ** -22 * size + UNIT[w[k].dtype] * np.linalg.norm(want[i])
    # in place: the same bits
    versions = [x._version for x in w + m]
    assert mk.orthogonal_step(w, g, m, 0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1)[0] is not None
    assert all(torch.equal(x, y) for x, y in zip(w + m, outs + kept))
    assert all(x._version > v for x, v in zip(w + m, versions))


def test_step_of_one_tensor_and_given_scales():
    gen = generator(5)
    g, m = gradient(gen, (64, 48)), gradient(gen, (64, 48))
    w = torch.zeros(64, 48, device="cuda")
    kept = torch.empty_like(m)
    mk.orthogonal_step(w, g, m, 1.0, momentum=0.5, nesterov=False, scale=2.0, momenta_outs=kept)
    o = mk.orthogonalize(0.5 * m + g)
    assert torch.allclose(w, -2.0 * o, rtol=1e-5, atol=1e-6)
    a, b = torch.zeros_like(w), torch.zeros_like(w)
    mk.orthogonal_step([a, b], [g, g], [m, m], 1.0, momentum=0.5, nesterov=False, scale=[2.0, 4.0],
                       momenta_outs=[kept, torch.empty_like(m)])
    assert torch.equal(a, w) and torch.equal(b, 2.0 * w)


def test_streams_and_graphs():
    gen = generator(6)
    gs = [gradient(gen, (200, 150)), gradient(gen, (100, 300))]
    want = mk.orthogonalize(gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mk.orthogonalize(gs, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    outs = [torch.zeros_like(g) for g in gs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.orthogonalize(gs, outs=outs)
    new = [gradient(gen, (200, 150)), gradient(gen, (100, 300))]
    for g, h in zip(gs, new):
        g.copy_(h)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, mk.orthogonalize(new)))


def test_refusals():
    x = torch.ones(6, 4, device="cuda")
    for kind, bad in [
            (TypeError, lambda: mk.orthogonalize(x.double())), (TypeError, lambda: mk.orthogonalize(x, dtype=torch.int32)),
            (ValueError, lambda: mk.orthogonalize([])), (ValueError, lambda: mk.orthogonalize(x[0])),
            (ValueError, lambda: mk.orthogonalize(x[::2, ::2])), (ValueError, lambda: mk.orthogonalize(x, outs=x[:3])),
            (ValueError, lambda: mk.orthogonalize(x, 3, [mk.QUINTIC] * 2)),
            (ValueError, lambda: mk.orthogonalize([x], scale=[1.0, 2.0])),
            (ValueError, lambda: mk.orthogonalize(torch.ones(2, 3, 4, 4, device="cuda")[:, :2])),
            (ValueError, lambda: mk.orthogonalize(x, outs=torch.ones(4, 6, device="cuda").mT)),
            (mk.MttkrpError, lambda: mk.orthogonalize(x, 0)), (mk.MttkrpError, lambda: mk.orthogonalize(x, 65)),
            (mk.MttkrpError, lambda: mk.orthogonalize(x, 5, (16.0, 0.0, 0.0))),
            (mk.MttkrpError, lambda: mk.orthogonalize(x, 5, (4.0, 0.0, 0.0))),
            (mk.MttkrpError, lambda: mk.orthogonalize(x, eps=-1.0)),
            (mk.MttkrpError, lambda: mk.orthogonalize([x, x], outs=[x, x])),
            (mk.MttkrpError, lambda: mk.orthogonalize([x, x], outs=[x, torch.ones_like(x)])),
            (mk.MttkrpError, lambda: mk.orthogonalize(x[:1].expand(6, 4))),
            (mk.MttkrpError, lambda: mk.orthogonal_step(x, x, x, 0.1)),
            (ValueError, lambda: mk.orthogonal_step([x], [x, x], [x], 0.1)),
            (TypeError, lambda: mk.orthogonal_step(x, x.cpu(), x, 0.1))]:
        with pytest.raises(kind):
            bad()
    assert torch.equal(x, torch.ones(6, 4, device="cuda"))


@pytest.mark.parametrize("weights,grads,momenta", MOMENTA)
@pytest.mark.parametrize("rows,cols,ahead", [(201, 333, 0), (333, 201, 3), (150, 264, 1), (264, 150, 0), (130, 136, 8)])
def test_step_at_odd_offsets(rows, cols, ahead, weights, grads, momenta):
    """Matrices with sides above 128 whose rows lie at any offset (and, in the last shape, aligned), in parts of
    wider ones: the new weight is the old one and the update, each rounded as the formula says."""
    gen = generator(rows + cols)

    def part(x, dtype):
        room = torch.full((rows, ahead + cols + 2), 3.0, device="cuda", dtype=dtype)
        view = room[:, ahead:ahead + cols]
        view.copy_(x)
        return room, view

    room_g, g = part(gradient(gen, (rows, cols)).mul(1e-3), TYPES[grads])
    room_m, m = part(gradient(gen, (rows, cols)).mul(5e-3), TYPES[momenta])
    room_w, w = part(torch.randn(rows, cols, generator=gen, device="cuda").mul(0.02), TYPES[weights])
    before_w, before_m, before_g = f64(w), f64(m), f64(g)
    by = max(1.0, rows / cols) ** 0.5
    mk.orthogonal_step(w, g, m, 0.02, momentum=0.9, weight_decay=0.1)
    want, want_m = oo.step(before_w, before_g, before_m, 0.02, 0.9, True, 0.1, by, 5, mk.QUINTIC)
    size = 0.9 * np.abs(before_m) + np.abs(before_g)
    assert np.all(np.abs(f64(m) - want_m) <= 2.0 ** -23 * size + UNIT[m.dtype] * 1.01 * np.abs(want_m) + 2.0 ** -25)
    u = before_g + 0.9 * (0.9 * before_m + before_g)
    bound, o = trajectory_bound(u, 5, mk.QUINTIC, 2.0 ** -11 if weights == "bfloat16" else 2.0 ** -20)
    bound += 4.25 ** 5 * 2.0 ** -23
    size = np.linalg.norm(before_w) + 0.02 * by * np.linalg.norm(o)
    err = np.linalg.norm(f64(w) - want)
    assert err <= 0.02 * by * bound + 2.0 ** -22 * size + UNIT[w.dtype] * np.linalg.norm(want)
    # each element near its own, so that none is misplaced: half of what 2 % of an update's typical element is
    typical = 0.02 * by / np.sqrt(max(rows, cols))
    assert np.abs(f64(w) - want).max() <= 0.5 * typical + UNIT[w.dtype] * 1.01 * np.abs(want).max()
    assert np.array_equal(f64(g), before_g)
    for room in (room_g, room_m, room_w):
        assert (room[:, :ahead] == 3).all() and (room[:, ahead + cols:] == 3).all()
