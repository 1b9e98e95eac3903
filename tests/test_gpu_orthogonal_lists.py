"""GPU orthogonalisation of lists of unlike matrices, whose products are dealt out together: every
matrix as the formula says, whatever else is in its call.

Whole numbers as in the tests of single matrices: G of 4^q entries +-1 has the norm 2^q, and S and S X are
whole numbers over powers of two, exact in the parts' bits and in the sums, so that results are
compared bit by bit after one rounding to their type."""
import numpy as np
import pytest

from oracle import orthogonal as oo

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def signs(seed, rows, cols, q):
    """4^q entries +-1, the others 0."""
    rng = np.random.default_rng(seed)
    g = np.zeros(rows * cols)
    g[rng.choice(rows * cols, 4 ** q, replace=False)] = rng.choice([-1.0, 1.0], 4 ** q)
    return g.reshape(rows, cols)


def cuda(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


# a long matrix, whose S is split over the CTAs of a cluster, with ones of three steps
UNLIKE = [[(512, 2000), (160, 160)], [(2000, 150), (150, 150), (150, 150)], [(768, 1024), (192, 192)],
          [(2500, 160), (160, 160)], [(512, 4096), (150, 150)], [(256, 1000), (129, 192), (192, 130)],
          [(192, 4097)], [(130, 2600), (257, 192), (129, 129)]]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shapes", UNLIKE)
def test_lists_of_unlike_matrices(shapes, dtype):
    gs = [signs(k, *s, 6) for k, s in enumerate(shapes)]
    got = mk.orthogonalize([cuda(g) for g in gs], 1, (0.0, 1.0, 0.0), eps=0.0, dtype=TYPES[dtype])
    assert mk.device_status() == 0
    for g, x in zip(gs, got):
        want = oo.orthogonalize(g, 1, (0.0, 1.0, 0.0), 0.0)
        assert torch.equal(x, cuda(want).to(TYPES[dtype])), g.shape


@pytest.mark.parametrize("shapes", UNLIKE)
def test_steps_of_unlike_matrices(shapes):
    """The training step takes the same path: weights of zero become -lr O(G), here of S X."""
    gs = [signs(k, *s, 6) for k, s in enumerate(shapes)]
    ws = [torch.zeros(*s, device="cuda") for s in shapes]
    ms = [torch.zeros(*s, device="cuda") for s in shapes]
    mk.orthogonal_step(ws, [cuda(g) for g in gs], ms, 1.0, momentum=0.5, nesterov=False, steps=1,
                       coefficients=(0.0, 1.0, 0.0), eps=0.0, scale=1.0)
    assert mk.device_status() == 0
    for g, w, m in zip(gs, ws, ms):
        assert torch.equal(w, cuda(-oo.orthogonalize(g, 1, (0.0, 1.0, 0.0), 0.0))) and torch.equal(m, cuda(g))


@pytest.mark.parametrize("eps", [0.0, 1e-300, 1e-80, 1e-7])
@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_stay_zeros(dtype, eps):
    """Whatever eps is, in both kinds of kernels and beside others; and the smallest number of each type is not zero."""
    shapes = [(65, 30), (30, 700), (128, 128), (130, 129), (200, 300)]
    gs = [torch.zeros(s, device="cuda", dtype=TYPES[dtype]) for s in shapes] + [cuda(signs(1, 140, 150, 3), TYPES[dtype])]
    got = mk.orthogonalize(gs, eps=eps)
    assert all(not x.any() for x in got[:-1]) and torch.isfinite(got[-1]).all() and got[-1].any()
    ws = [torch.ones_like(g) for g in gs]
    mk.orthogonal_step(ws, gs, [torch.zeros_like(g) for g in gs], 0.5, eps=eps)
    assert all((w == 1).all() for w in ws[:-1]) and torch.isfinite(ws[-1]).all()
    least = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}[dtype]
    for shape in ((20, 33), (130, 150)):
        g = torch.zeros(shape, device="cuda", dtype=TYPES[dtype])
        g[3, 7] = least
        x = mk.orthogonalize(g, 1, (1.0, 0.0, 0.0), eps=0.0)
        assert x[3, 7] == 1 and x.sum() == 1


UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# relative (Frobenius norm) errors of five quintic steps before the result's rounding, as include/mttkrp.h says:
# products of 22 bits, and of 11 (but for X) where a result in bf16 has both sides above 128
LONG, SHORT = 4e-6, 1.5e-3


def gradient(gen, shape, dtype):
    """A few strong directions over noise."""
    r, c = shape
    rank = max(1, min(r, c) // 16)
    u = torch.randn(r, rank, generator=gen, device="cuda")
    v = torch.randn(rank, c, generator=gen, device="cuda")
    return (u @ v / rank ** 0.5 + 0.1 * torch.randn(r, c, generator=gen, device="cuda")).to(dtype)


SIDES = [(90, 70), (33, 47), (257, 128), (70, 301), (256, 64), (129, 130), (201, 333), (501, 333), (512, 2000), (1100, 900),
         (2048, 700)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SIDES)
def test_results_as_near_as_promised(shape, dtype):
    """A rounding moves a value by half a step of its type at most, and so the whole by no more of its norm; fp16's
    smallest numbers by 2^-25 each."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    g = gradient(gen, shape, TYPES[dtype])
    want = oo.orthogonalize(g.double().cpu(), 5, mk.QUINTIC)
    size = np.linalg.norm(want)
    short = dtype == "bfloat16" and min(shape) > 128
    bound = (SHORT if short else LONG) + UNIT[TYPES[dtype]] + (2.0 ** -25 * want.size ** 0.5 / size if dtype == "float16" else 0)
    x = mk.orthogonalize(g)
    assert np.linalg.norm(x.double().cpu().numpy() - want) <= bound * size
    # into fp32, whatever the input's type: nothing but the products
    x = mk.orthogonalize(g, dtype=torch.float32)
    assert np.linalg.norm(x.double().cpu().numpy() - want) <= (LONG + UNIT[torch.float32]) * size


@pytest.mark.parametrize("weights", TYPES)
@pytest.mark.parametrize("momenta", TYPES)
@pytest.mark.parametrize("shape", SIDES)
def test_updates_as_near_as_promised(shape, weights, momenta):
    """What a step adds to weights of zeros: -lr scale O(U), U within two roundings of fp32 (4e-6 after five
    steps: a direction a hundredth as strong as the whole is raised to 1 by up to 485, and its rounding with it)."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape) + 1)
    g, m = gradient(gen, shape, torch.bfloat16), gradient(gen, shape, TYPES[momenta])
    w = torch.zeros(shape, device="cuda", dtype=TYPES[weights])
    before = m.double().cpu().numpy()
    mk.orthogonal_step(w, g, m, 0.5, momentum=0.9, scale=2.0)
    kept = 0.9 * before + g.double().cpu().numpy()
    want = -oo.orthogonalize(g.double().cpu().numpy() + 0.9 * kept, 5, mk.QUINTIC)
    size = np.linalg.norm(want)
    short = weights == "bfloat16" and min(shape) > 128
    bound = (SHORT if short else LONG) + 4e-6 + UNIT[w.dtype] + (2.0 ** -25 * want.size ** 0.5 / size if weights == "float16" else 0)
    assert np.linalg.norm(w.double().cpu().numpy() - want) <= bound * size
    assert np.all(np.abs(m.double().cpu().numpy() - kept) <= 2.0 ** -23 * (np.abs(before) + np.abs(kept)) * 2 +
                  UNIT[m.dtype] * 1.01 * np.abs(kept) + (2.0 ** -25 if momenta == "float16" else 0))


@pytest.mark.parametrize("shape", [(64, 64), (64, 6000), (128, 512), (129, 130), (512, 512), (2000, 512), (1024, 1100)])
@pytest.mark.parametrize("abc", [mk.QUINTIC, (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8)])
def test_sums_of_mixed_signs(shape, abc):
    """One step of normal numbers, whose sums of P X have both signs and are led by the diagonal's term: the
    parts of X and P are within 2^-23 of them; what is put back for additions that are cut off is 2.4e-7
    (128 indices) at most, and never more off than that where they lose less; S and S S, of which P is a small
    share beside a I, with the same errors: less than half as much again."""
    gen = torch.Generator(device="cuda").manual_seed(shape[0])
    g = torch.randn(shape, generator=gen, device="cuda")
    want = oo.orthogonalize(g.double().cpu(), 1, abc, 0.0)
    x = mk.orthogonalize(g, 1, abc, eps=0.0).double().cpu().numpy()
    off = x - want
    size = np.linalg.norm(want)
    assert np.linalg.norm(off) <= 1.5 * (2 * 2.0 ** -23 + 2.4e-7) * size
    assert abs((off * want).sum()) <= 2.4e-7 * size ** 2


@pytest.mark.parametrize("noise", [1.0, 0.1, 1e-3])
@pytest.mark.parametrize("shape", [(64, 300), (20, 128), (128, 1000), (128, 1833), (64, 6000), (70, 2900), (129, 130), (200, 200),
                                   (333, 501), (1024, 256), (900, 1100)])
def test_no_more_than_twice_as_far_as_fp32(shape, noise):
    """Five steps, weak directions of several sizes: twice the error of fp32 products is what is documented."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    r, c = shape
    rank = max(1, min(r, c) // 16)
    u = torch.randn(r, rank, generator=gen, device="cuda")
    v = torch.randn(rank, c, generator=gen, device="cuda")
    g = u @ v / rank ** 0.5 + noise * torch.randn(r, c, generator=gen, device="cuda")
    want = oo.orthogonalize(g.double().cpu(), 5, mk.QUINTIC)
    torch.backends.cuda.matmul.allow_tf32 = False
    x = g / (g.norm() + 1e-7)
    x = x.mT if r > c else x
    for _ in range(5):
        s = x @ x.mT
        x = mk.QUINTIC[0] * x + (mk.QUINTIC[1] * s + mk.QUINTIC[2] * (s @ s)) @ x
    x = x.mT if r > c else x
    plain = np.linalg.norm(x.double().cpu().numpy() - want)
    here = np.linalg.norm(mk.orthogonalize(g).double().cpu().numpy() - want)
    assert here <= max(2 * plain, 1e-6 * np.linalg.norm(want))
