"""GPU row lookups, CP model entries, their gradients and clipping, through the
binding and the C ABI, against the fp64 oracle on the same inputs.

Bounds (u = 2^-24, the unit roundoff of fp32; v that of the result's type): a sum
of k fp32 terms, each with j roundings of its own, is within (k + j) u times the sum
of the terms' magnitudes of the exact one, whatever the order; rounding the result
adds v of its magnitude, or half the type's smallest step below its normal range."""
import numpy as np
import pytest

from oracle import sampled as os_

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
UNIT = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEP = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def f64(t):
    return t.double().cpu().numpy()


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tokens(gen, n, rows, skew=1.0, masked=0.05, dtype=torch.int64):
    """n indices, some of them -1, rows or beyond."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    idx = (rows * u ** skew).long().clamp_(max=rows - 1)
    r = torch.rand(n, generator=gen, device="cuda")
    idx = torch.where(r < masked / 3, -1, idx)
    idx = torch.where((r >= masked / 3) & (r < 2 * masked / 3), rows, idx)
    idx = torch.where((r >= 2 * masked / 3) & (r < masked), rows + 1000003, idx)
    return idx.to(dtype)


# ---------------------------------------------------------------- lookup

LOOKUPS = [(1, 1, 1), (1, 7, 2000), (2, 5, 3), (31, 40, 8), (33, 512, 64), (257, 100, 1001), (1000, 32, 17),
           (4099, 3000, 256), (130, 9, 4096), (64, 50, 65536),
           (3001, 70, 5), (700, 90, 159), (701, 90, 161), (333, 20, 255), (555, 30, 257), (90, 8, 2), (5000, 9, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,rows,width", LOOKUPS)
def test_lookup_is_one_product_and_one_rounding(n, rows, width, dtype):
    gen = generator(n + rows + width)
    table = normal(gen, (rows, width), TYPES[dtype])
    idx = tokens(gen, n, rows, dtype=torch.int32 if n % 2 else torch.int64)
    out = mk.embedding(table, idx, scale=0.37)
    assert out.shape == (n, width) and out.dtype == table.dtype
    i = idx.cpu().long()
    inside = (i >= 0) & (i < rows)
    want = (table.cpu()[i.clamp(0, rows - 1)].float() * torch.tensor(0.37)).to(table.dtype)
    assert torch.equal(out.cpu(), torch.where(inside[:, None], want, torch.zeros((), dtype=table.dtype)))


def test_lookup_strides_shapes_and_offsets():
    gen = generator(3)
    big = normal(gen, (50, 80), torch.float32)
    coords = torch.randint(0, 50, (77, 3), generator=gen, device="cuda")
    for cols in (slice(0, 64), slice(3, 64), slice(1, 2), slice(4, 36)):     # rows 320 bytes apart, any start
        table = big[:, cols]
        width = table.shape[1]
        for idx in (coords[:, 1], coords[:, 1].contiguous(), coords):
            out = mk.embedding(table, idx, scale=2.0)
            assert torch.equal(out, 2.0 * table[idx])
            room = torch.zeros((coords[:, 0].numel() * 3, width + 5), device="cuda")
            if idx.dim() == 1:
                dst = room[:77, 2:2 + width]
                assert mk.embedding(table, idx, scale=2.0, out=dst).data_ptr() == dst.data_ptr()
                assert torch.equal(dst, 2.0 * table[idx])
                assert room[:, :2].abs().sum() == 0 and room[77:].abs().sum() == 0
                assert room[:, 2 + width:].abs().sum() == 0
    assert mk.embedding(big, coords[:0, 0]).shape == (0, 80)
    assert mk.embedding(big, coords[:1, 0].expand(6)).shape == (6, 80)       # one index, stride 0
    assert mk.embedding(big, torch.tensor(7, device="cuda")).shape == (80,)


def test_lookup_leaves_masked_rows_unread():
    table = torch.full((4, 33), float("nan"), device="cuda")
    table[1] = 5.0
    idx = torch.tensor([1, -1, 4, 1 << 40, -(1 << 40), (1 << 32) + 1], device="cuda")
    out = mk.embedding(table, idx)
    assert torch.equal(out[0], table[1]) and out[1:].abs().sum() == 0
    inf = torch.full((1, 8), float("inf"), device="cuda")
    assert torch.isinf(mk.embedding(inf, idx[:1] * 0)).all()


# ---------------------------------------------------------------- gradient of the lookup

def check_grad(idx, grad, rows, scale, got, before=None):
    i, g = idx.cpu().numpy().reshape(-1), f64(grad).reshape(idx.numel(), grad.shape[-1])
    want = os_.embedding_grad(i, g, rows, scale)
    mag = os_.embedding_grad(i, np.abs(g), rows, abs(scale))
    count = np.bincount(i[(i >= 0) & (i < rows)], minlength=rows)[:, None]
    if before is not None:
        want, mag = want + before, mag + np.abs(before)
        untouched = np.broadcast_to(count == 0, want.shape)
        assert np.array_equal(f64(got)[untouched], before[untouched])
    bound = (count + 3) * U * mag + UNIT[got.dtype] * np.abs(want) * 1.01 + STEP[got.dtype]
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), (err - bound).max()
    if before is None:
        assert np.all(f64(got)[(count == 0)[:, 0]] == 0)


GRADS = [  # tokens, rows, width, skew
    (0, 5, 3, 1), (1, 1, 1, 1), (1, 700, 2000, 1), (2, 3, 8, 1), (7, 5, 100, 1), (8, 4, 33, 1), (9, 1, 64, 1),
    (31, 40, 17, 1), (48, 512, 256, 1), (257, 2, 40, 1), (1000, 1, 24, 1), (1025, 1023, 12, 1), (1500, 1024, 8, 1),
    (5003, 300, 65, 2), (8191, 70000, 16, 1), (8192, 50, 128, 3), (8193, 50, 72, 3), (20011, 3, 40, 1),
    (33000, 33000, 9, 1), (70001, 1 << 20, 4, 2), (100003, 513, 32, 4), (300007, 5000, 8, 3), (40, 9, 65536, 1),
    (30000, 700, 38, 2), (777, 50, 90, 1)]


@pytest.mark.parametrize("n,rows,width,skew", GRADS)
@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "float32"), ("bfloat16", "bfloat16"),
                                       ("float16", "float32"), ("float16", "float16")])
def test_lookup_gradient(n, rows, width, skew, dtype, out):
    gen = generator(7 * n + rows + width)
    idx = tokens(gen, n, rows, skew, dtype=torch.int32 if n % 2 else torch.int64)
    grad = normal(gen, (n, width), TYPES[dtype])
    got = mk.embedding_grad(idx, grad, rows, scale=-0.75, dtype=TYPES[out])
    assert got.shape == (rows, width) and got.dtype == TYPES[out]
    check_grad(idx, grad, rows, -0.75, got)
    assert torch.equal(got, mk.embedding_grad(idx, grad, rows, scale=-0.75, dtype=TYPES[out]))


@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "float32"), ("float16", "float16")])
@pytest.mark.parametrize("n,rows,width", [(0, 6, 5), (1, 3, 4), (300, 7, 40), (5000, 400, 33), (9000, 20, 64)])
def test_lookup_gradient_added_to_what_is_there(n, rows, width, dtype, out):
    gen = generator(n + 11)
    idx = tokens(gen, n, rows)
    grad = normal(gen, (n, width), TYPES[dtype])
    acc = normal(gen, (rows, width), TYPES[out])
    before = f64(acc)
    assert mk.embedding_grad(idx, grad, rows, scale=0.5, out=acc, accumulate=True) is acc
    check_grad(idx, grad, rows, 0.5, acc, before)


@pytest.mark.parametrize("offset,width,pad", [(0, 64, 8), (1, 64, 7), (4, 40, 24), (0, 33, 0), (0, 96, 32)])
def test_lookup_gradient_strides_and_offsets(offset, width, pad):
    """Column slices of wider buffers; what lies between the rows stays."""
    gen = generator(offset + width)
    coords = torch.randint(-1, 30, (3000, 2), generator=gen, device="cuda", dtype=torch.int32)
    wide = normal(gen, (3000, offset + width + pad), torch.bfloat16)
    grad = wide[:, offset:offset + width]
    for dt in (torch.float32, torch.bfloat16):
        room = torch.full((31, offset + width + pad), 7.0, device="cuda", dtype=dt)
        out = room[:, offset:offset + width]
        got = mk.embedding_grad(coords[:, 1], grad, 31, out=out)
        check_grad(coords[:, 1], grad, 31, 1.0, got)
        assert torch.all(room[:, :offset] == 7.0) and torch.all(room[:, offset + width:] == 7.0)


def test_lookup_gradient_masks_leave_nothing():
    """Every token masked; NaN and infinities in masked gradients; a NaN in a kept one stays in its row."""
    grad = torch.full((500, 36), float("nan"), device="cuda")
    idx = torch.full((500,), -1, device="cuda")
    assert mk.embedding_grad(idx, grad, 9).abs().sum() == 0
    acc = torch.ones((9, 36), device="cuda")
    mk.embedding_grad(idx, grad, 9, out=acc, accumulate=True)
    assert torch.all(acc == 1)
    idx[17] = 4
    idx[18] = 4
    grad[17] = 1.5
    grad[18] = 2.0
    got = mk.embedding_grad(idx, grad, 9)
    assert torch.all(got[4] == 3.5) and got[:4].abs().sum() == 0 and got[5:].abs().sum() == 0
    idx[30] = 2
    grad[30, 3] = float("inf")
    got = mk.embedding_grad(idx, grad, 9)
    assert torch.isnan(got[2]).sum() == 35 and torch.isinf(got[2, 3]) and torch.all(got[4] == 3.5)


# ---------------------------------------------------------------- CP model

MODELS = [  # dims, R, samples
    ((5,), 3, 40), ((1, 1), 1, 7), ((6, 7), 8, 1), ((32, 32, 32), 8, 1000), ((9, 4, 7), 33, 500),
    ((20,) * 6, 128, 3001), ((300, 2, 50), 64, 5000), ((2,) * 8, 20, 2000), ((40, 50, 60), 257, 700),
    ((512, 1, 3), 100, 9001), ((64, 64, 64), 2000, 130), ((1500, 1100), 16, 20000), ((7, 8, 9), 4, 0),
    # more samples than one CTA groups, factors that fit shared memory in slices of 32, 16 and 8 columns or
    # not at all, as tables of single modes and of products, ranks that end inside a slice
    ((20,) * 5 + (21,), 128, 40001), ((512, 512, 513), 96, 50000), ((40, 50, 60), 257, 30000),
    ((1000, 900, 800), 48, 33000), ((2000, 1500, 1900), 20, 33001), ((3,) * 8, 36, 20003), ((30, 17), 1, 17000),
    ((100003, 9, 4), 24, 40000), ((9,), 33, 25000), ((5, 1, 1, 1, 1, 1, 1), 12, 18000), ((250, 250), 1000, 17001),
    # five to eight tables a sample, the same number for every mode and not
    ((48,) * 6, 40, 20000), ((41,) * 8, 17, 17003), ((200, 3, 150, 70, 2, 90, 5), 36, 24001),
    ((700, 900, 600, 30, 30, 20, 40), 8, 30000), ((45,) * 5, 64, 18000)]


def coords_of(gen, dims, S, dtype=torch.int32, masked=0.05):
    c = torch.stack([tokens(gen, S, n, masked=masked) for n in dims], dim=1)
    return c.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dims,R,S", MODELS)
def test_entries(dims, R, S, dtype):
    gen = generator(sum(dims) + R + S)
    A = [normal(gen, (n, R), TYPES[dtype]) for n in dims]
    c = coords_of(gen, dims, S, torch.int64 if S % 2 else torch.int32)
    got = mk.cp_entries(A, c)
    A64, cn = [f64(a) for a in A], c.cpu().numpy()
    want = os_.cp_entries(A64, cn)
    mag = os_.cp_entries([np.abs(a) for a in A64], cn)
    assert got.shape == (S,) and got.dtype == torch.float32
    assert np.all(np.abs(f64(got) - want) <= (R + len(dims)) * U * mag)
    assert torch.equal(got, mk.cp_entries(A, c))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dims,R,S", MODELS)
def test_entries_gradient(dims, R, S, dtype):
    gen = generator(sum(dims) + R + S + 1)
    A = [normal(gen, (n, R), TYPES[dtype]) for n in dims]
    c = coords_of(gen, dims, S, torch.int64 if S % 2 else torch.int32)
    g = normal(gen, (S,), torch.float32)
    got = mk.cp_entries_grad(A, c, g)
    A64, cn, g64 = [f64(a) for a in A], c.cpu().numpy(), f64(g)
    want = os_.cp_entries_grad(A64, cn, g64)
    mag = os_.cp_entries_grad([np.abs(a) for a in A64], cn, np.abs(g64))
    inside = ((cn >= 0) & (cn < np.array(dims))).all(axis=1)
    for n, G in enumerate(got):
        assert G.shape == (dims[n], R) and G.dtype == torch.float32
        count = np.bincount(cn[inside, n], minlength=dims[n])[:, None]
        err = np.abs(f64(G) - want[n])
        assert np.all(err <= (count + len(dims) + 1) * U * mag[n] + 2.0 ** -149), n
    for a, b in zip(got, mk.cp_entries_grad(A, c, g)):
        assert torch.equal(a, b)


def test_entries_gradient_matches_differences():
    """<G, direction> against the change of <g, entries> along it (fp64 entries)."""
    gen = generator(77)
    dims, R, S = (12, 9, 15), 10, 400
    A = [normal(gen, (n, R), torch.float32) for n in dims]
    c, g = coords_of(gen, dims, S), normal(gen, (S,), torch.float32)
    G = mk.cp_entries_grad(A, c, g)
    h = 1e-4
    for n in range(3):
        D = np.random.default_rng(n).standard_normal((dims[n], R))
        up, down = [f64(a) for a in A], [f64(a) for a in A]
        up[n], down[n] = up[n] + h * D, down[n] - h * D
        cn = c.cpu().numpy()
        diff = np.sum(f64(g) * (os_.cp_entries(up, cn) - os_.cp_entries(down, cn))) / (2 * h)
        # the entries are linear in one factor: the difference is exact up to fp64 rounding
        scale = np.sum(np.abs(f64(G[n])) * np.abs(D))
        assert abs(np.sum(f64(G[n]) * D) - diff) <= (S + 4) * U * scale + 1e-9 * scale


def test_masked_samples_read_nothing():
    dims, R = (4, 5, 6), 40
    A = [torch.full((n, R), float("nan"), device="cuda") for n in dims]
    for a in A:
        a[1] = 2.0
    c = torch.tensor([[1, 1, 1], [-1, 1, 1], [1, 5, 1], [0, 0, 6], [1, 1, -7]], device="cuda", dtype=torch.int32)
    g = torch.tensor([1.0, float("nan"), float("inf"), float("nan"), 3.0], device="cuda")
    x = mk.cp_entries(A, c)
    assert x.tolist() == [8.0 * R, 0.0, 0.0, 0.0, 0.0]
    for n, G in enumerate(mk.cp_entries_grad(A, c, g)):
        assert torch.all(G[1] == 4.0) and G.abs().sum() == 4.0 * R


def test_weights_as_a_factor_with_one_row():
    gen = generator(5)
    A = [normal(gen, (n, 24), torch.float32) for n in (30, 20)]
    lam = torch.rand(24, generator=gen, device="cuda")
    c = coords_of(gen, (30, 20), 2500, masked=0.0)
    one = torch.cat([c, torch.zeros_like(c[:, :1])], dim=1)
    got = mk.cp_entries(A + [lam[None]], one)
    want = os_.cp_entries([f64(A[0]) * f64(lam), f64(A[1])], c.cpu().numpy())
    assert np.allclose(f64(got), want, rtol=0, atol=30 * U * np.abs(want).max() * 24)
    g = normal(gen, (2500,), torch.float32)
    G = mk.cp_entries_grad(A + [lam[None]], one, g)[2]
    rows = f64(A[0])[c[:, 0].cpu()] * f64(A[1])[c[:, 1].cpu()]
    want = (f64(g)[:, None] * rows).sum(0)
    assert np.all(np.abs(f64(G)[0] - want) <= 2504 * U * (np.abs(f64(g)[:, None]) * np.abs(rows)).sum(0))


# ---------------------------------------------------------------- norm and clipping

def check_clip(ts, max_norm, eps, norm, ys):
    """The norm: at most 16 fp32 roundings a square's group, half of that under the
    root, one more at the end; the coefficient follows it; one product, one rounding."""
    want, clipped = os_.clip([f64(t) for t in ts], max_norm, eps)
    assert abs(float(norm) - want) <= 10 * U * want
    for t, y, w in zip(ts, ys, clipped):
        assert y.dtype == t.dtype
        err = np.abs(f64(y) - w.reshape(y.shape))
        assert np.all(err <= (14 * U + UNIT[t.dtype]) * np.abs(w.reshape(y.shape)) * 1.01 + STEP[t.dtype])


SETS = [[1], [0], [5, 0, 3], [7, 1, 4097, 16384, 16385], [100003], [3, 0, 0, 2, 1 << 20],
        [1 + (k * 37) % 501 for k in range(40)], [k % 19 for k in range(1100)], [262144 + 5] * 3, [64] * 2500]


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dtype", [*TYPES, "mixed"])
def test_norm_and_clipping(sizes, dtype):
    gen = generator(len(sizes) + sum(sizes))
    kinds = list(TYPES.values())
    ts = [normal(gen, (n,), kinds[k % 3] if dtype == "mixed" else TYPES[dtype], 0.1) for k, n in enumerate(sizes)]
    norm = mk.grad_norm(ts)
    assert norm.dtype == torch.float32 and norm.shape == ()
    true = np.sqrt(sum(np.sum(f64(t) ** 2) for t in ts))
    for max_norm in (0.3 * true, 3.0 * true + 1.0):
        outs = [torch.full_like(t, 9.0) for t in ts]
        got = mk.clip_grad_norm(ts, max_norm, outs=outs)
        assert torch.equal(got, norm)
        check_clip(ts, max_norm, 1e-6, got, outs)
        own = [t.clone() for t in ts]
        assert torch.equal(mk.clip_grad_norm(own, max_norm), norm)
        assert all(torch.equal(a, b) for a, b in zip(own, outs))


@pytest.mark.parametrize("dtype", TYPES)
def test_clipping_of_views_at_any_offset(dtype):
    """Packed views of one buffer, in and out at different offsets; the gaps stay."""
    gen = generator(8)
    sizes = [1, 5, 1000, 3, 40000, 77, 16384]
    flat = normal(gen, (sum(sizes) + 20,), TYPES[dtype])
    room = torch.full((sum(sizes) + 40,), 3.0, device="cuda", dtype=TYPES[dtype])
    for shift in (0, 1, 2, 7):
        room.fill_(3.0)
        ts, outs, at, to = [], [], 3, 3 + shift
        for n in sizes:
            ts.append(flat[at:at + n])
            outs.append(room[to:to + n])
            at, to = at + n, to + n + 1
        norm = mk.clip_grad_norm(ts, 1.5, outs=outs)
        check_clip(ts, 1.5, 1e-6, norm, outs)
        used = torch.zeros_like(room, dtype=torch.bool)
        to = 3 + shift
        for n in sizes:
            used[to:to + n] = True
            to += n + 1
        assert torch.all(room[~used] == 3.0)


def test_norm_outside_the_range_of_fp32_squares():
    """Squares that overflow or vanish in fp32 do not in the norm; zeros stay zero."""
    for value in (1e30, 3e19, 1e-30, 1e-42, 2.0 ** -149):
        t = torch.full((1001,), value, device="cuda")
        want = float(t[0].double()) * np.sqrt(1001.0)
        got = float(mk.grad_norm([t, torch.zeros(50000, device="cuda")]))
        assert abs(got - want) <= 10 * U * want + 2.0 ** -149, value
    mix = torch.tensor([1e-30] * 100 + [1e25] + [0.0] * 500, device="cuda")
    assert abs(float(mk.grad_norm([mix])) - 1e25) <= 1e25 * 10 * U
    z = [torch.zeros(3, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(mk.clip_grad_norm(z, 1.0)) == 0.0 and z[0].tolist() == [0.0, 0.0, 0.0]


def test_norms_that_are_not_finite_follow_the_formula():
    t = torch.ones(100, device="cuda")
    t[3] = float("inf")
    y = torch.empty_like(t)
    assert float(mk.clip_grad_norm([t], 1.0, outs=[y])) == float("inf")
    assert y.isnan().sum() == 1 and torch.isnan(y[3]) and y[0] == 0      # 0 * inf, 0 * 1
    t[3] = float("nan")
    assert np.isnan(float(mk.clip_grad_norm([t], 1.0, outs=[y]))) and torch.isnan(y).all()
    t[3] = 1.0
    assert float(mk.clip_grad_norm([t], 0.0)) == 10.0 and torch.all(t == 0)


# ---------------------------------------------------------------- all of them

def test_on_another_stream():
    """Everything enqueued on the stream that is given, or on the current one."""
    gen = generator(21)
    table = normal(gen, (300, 96), torch.float32)
    idx = tokens(gen, 4000, 300)
    A = [normal(gen, (n, 48), torch.float32) for n in (30, 40)]
    c = coords_of(gen, (30, 40), 4000)
    g = normal(gen, (4000,), torch.float32)

    def all_of(stream=None):
        rows = mk.embedding(table, idx, 3.0, stream=stream)
        G = mk.embedding_grad(idx, rows, 300, stream=stream)
        x = mk.cp_entries(A, c, stream=stream)
        H = mk.cp_entries_grad(A, c, g, stream=stream)
        norm = mk.clip_grad_norm([G, *H], 1.0, stream=stream)
        return [rows, G, x, *H, norm]

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        inside = all_of()
    torch.cuda.synchronize()
    given = all_of(stream=side)
    torch.cuda.synchronize()
    for a, b, d in zip(want, inside, given):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_replayed_from_a_graph():
    gen = generator(22)
    idx = tokens(gen, 9000, 500)
    grad = normal(gen, (9000, 64), torch.bfloat16)
    A = [normal(gen, (n, 32), torch.float32) for n in (30, 40)]
    c, g = coords_of(gen, (30, 40), 9000), normal(gen, (9000,), torch.float32)

    def step():
        G = mk.embedding_grad(idx, grad, 500)
        H = mk.cp_entries_grad(A, c, g)
        return [G, *H, mk.clip_grad_norm([G, *H], 0.5)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    grad.copy_(normal(gen, (9000, 64), torch.bfloat16))
    g.copy_(normal(gen, (9000,), torch.float32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    """Tables and gradients of more than 2^31 elements, read and written at their ends."""
    rows, width = 36000, 65536                                            # 2.36 Gi elements
    table = torch.zeros((rows, width), device="cuda", dtype=torch.bfloat16)
    idx = torch.tensor([rows - 1, 0, 32768, rows - 2, rows - 1, rows], device="cuda")
    for k in idx[:5].unique().tolist():
        table[k] = float(k % 97) + 1
    out = mk.embedding(table, idx)
    assert torch.equal(out[:5], table[idx[:5]]) and out[5].abs().sum() == 0
    table.fill_(1.0)
    got = mk.embedding_grad(idx, out, rows, out=table)
    assert got is table
    for k in range(5):
        twice = 2 if k in (0, 4) else 1
        assert torch.equal(table[idx[k]].float(), twice * out[k].float())
    kept = set(idx[:5].tolist())
    for lo in range(0, rows, 4000):
        part = table[lo:lo + 4000].float().abs().amax(dim=1)
        zero = [r for r in range(lo, min(rows, lo + 4000)) if r not in kept]
        assert part[torch.tensor(zero, device="cuda") - lo].sum() == 0
    norm = mk.grad_norm([table])
    want = np.sqrt(sum((2.0 if k in (0,) else 1.0) ** 2 * float(out[k].double().square().sum())
                       for k in (0, 1, 2, 3)))
    assert abs(float(norm) - want) <= 10 * U * want
    del table, out, got
    torch.cuda.empty_cache()


def test_refusals():
    f = torch.zeros((6, 8), device="cuda")
    i = torch.zeros(5, dtype=torch.int64, device="cuda")
    for bad in (lambda: mk.embedding(f.cpu(), i), lambda: mk.embedding(f, i.cpu()),
                lambda: mk.embedding(f.double(), i), lambda: mk.embedding(f, i.float()),
                lambda: mk.embedding_grad(i.short(), f[:5], 4), lambda: mk.cp_entries([f], i.float()[:, None]),
                lambda: mk.grad_norm([f, f.double()]), lambda: mk.clip_grad_norm([f, 3.0], 1.0),
                lambda: mk.cp_entries([f.long()], i[:, None])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: mk.embedding(f[0], i), lambda: mk.embedding(f.t(), i),
                lambda: mk.embedding(f, i[:4].view(2, 2).t()), lambda: mk.embedding(f, i, out=f[:5, :4]),
                lambda: mk.embedding(f, i, out=torch.zeros((5, 8), device="cuda").half()),
                lambda: mk.embedding_grad(i, f, 4), lambda: mk.embedding_grad(i, f[:5], 4, accumulate=True),
                lambda: mk.embedding_grad(i, f[:5], 4, out=torch.zeros((5, 8), device="cuda")),
                lambda: mk.embedding_grad(i, f[:5].t().contiguous().t(), 4),
                lambda: mk.cp_entries([f, f[:, :4]], torch.zeros((3, 2), dtype=torch.int32, device="cuda")),
                lambda: mk.cp_entries([f, f.half()], torch.zeros((3, 2), dtype=torch.int32, device="cuda")),
                lambda: mk.cp_entries([f], torch.zeros((3, 2), dtype=torch.int32, device="cuda")),
                lambda: mk.cp_entries([], i[:, None]), lambda: mk.cp_entries([f.t()], i[:, None]),
                lambda: mk.cp_entries([f], i[:, None], out=torch.zeros(4, device="cuda")),
                lambda: mk.cp_entries_grad([f], i[:, None], torch.zeros(4, device="cuda")),
                lambda: mk.cp_entries_grad([f], i[:, None], torch.zeros(5, device="cuda"), outs=[f[:5]]),
                lambda: mk.grad_norm([]), lambda: mk.grad_norm([f.t()]),
                lambda: mk.clip_grad_norm([f], 1.0, outs=[f.half()]), lambda: mk.clip_grad_norm([f], 1.0, outs=[])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mk.embedding_grad(i, f[:5], 0), lambda: mk.embedding(f, i, out=f[:5]),
                lambda: mk.embedding_grad(i, f[:5], 6, out=f), lambda: mk.clip_grad_norm([f], -1.0),
                lambda: mk.clip_grad_norm([f], float("nan")), lambda: mk.embedding_grad(i, f[:5].half(), 4, dtype=torch.bfloat16),
                lambda: mk.cp_entries_grad([f], i[:, None], torch.zeros(5, device="cuda"), outs=[f]),
                lambda: mk.clip_grad_norm([f.view(-1)[:40]], 1.0, outs=[f.view(-1)[1:41]]),
                lambda: mk.cp_entries([f] * 9, torch.zeros((3, 9), dtype=torch.int32, device="cuda"))):
        with pytest.raises(mk.MttkrpError):
            bad()
