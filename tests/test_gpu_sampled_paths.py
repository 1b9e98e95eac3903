"""GPU paths of the sampled operators that only large calls, large results or operands at
odd offsets take.

Values are small whole numbers, so that every product and sum is exact in fp32 (and in the
result's type) whatever the order: results must equal those in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(gen, shape, dtype, low=-3, high=4):
    return torch.randint(low, high, shape, generator=gen, device="cuda").to(dtype)


def tokens(gen, n, rows, skew=1.0, dtype=torch.int32):
    """n indices below `rows`, about 3 % of them outside."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    idx = (rows * u ** skew).long().clamp_(max=rows - 1)
    r = torch.rand(n, generator=gen, device="cuda")
    idx = torch.where(r < 0.015, -1, idx)
    return torch.where((r >= 0.015) & (r < 0.03), rows, idx).to(dtype)


def placed(flat_of, shape, offset):
    """A contiguous tensor of `shape` that starts `offset` elements into a buffer, and the buffer."""
    numel = 1
    for n in shape:
        numel *= n
    flat = flat_of(numel + offset + 16)
    return flat[offset:offset + numel].view(shape), flat


def sums_in_64_bits(idx, grad, rows):
    i = idx.long()
    kept = ((i >= 0) & (i < rows)).nonzero().flatten()
    out = torch.zeros((rows, grad.shape[1]), device="cuda", dtype=torch.float64)
    return out.index_add_(0, i[kept], grad[kept].double())


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan"), -2.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 2, 3, 8, 17, 33, 64, 65, 127, 130, 1001])
def test_masked_rows_are_zero_whatever_the_scale(width, dtype, scale):
    gen = generator(width)
    table = whole(gen, (20, width), TYPES[dtype], 1, 5)
    idx = torch.tensor([3, -1, 20, 19, 1 << 40, 0, -7], device="cuda").repeat(30)
    out = mk.embedding(table, idx, scale=scale)
    inside = (idx >= 0) & (idx < 20)
    bits = out[~inside].view(torch.int32 if dtype == "float32" else torch.int16)
    assert torch.all(bits == 0)                                          # +0
    want = (table[idx[inside]].float() * scale).to(table.dtype)
    assert torch.equal(out[inside].nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


def test_results_written_in_place_are_seen_by_autograd():
    gen = generator(2)
    table, idx = whole(gen, (9, 12), torch.float32), torch.tensor([1, 2, 8], device="cuda")
    A, c = [whole(gen, (n, 12), torch.float32) for n in (5, 6)], torch.zeros((3, 2), device="cuda", dtype=torch.int32)
    g = torch.ones(3, device="cuda")
    rows, sums, x = torch.empty((3, 12), device="cuda"), torch.empty((9, 12), device="cuda"), torch.empty(3, device="cuda")
    outs, scaled = [torch.empty_like(a) for a in A], torch.empty_like(table)
    for call, written, read in (
            (lambda: mk.embedding(table, idx, out=rows), [rows], [table, idx]),
            (lambda: mk.embedding_grad(idx, rows, 9, out=sums), [sums], [idx, rows]),
            (lambda: mk.embedding_grad(idx, rows, 9, out=sums, accumulate=True), [sums], [idx, rows]),
            (lambda: mk.cp_entries(A, c, out=x), [x], A),
            (lambda: mk.cp_entries_grad(A, c, g, outs=outs), outs, A + [g]),
            (lambda: mk.clip_grad_norm([table], 1.0, outs=[scaled]), [scaled], [table]),
            (lambda: mk.clip_grad_norm([table, sums], 1.0), [table, sums], []),
            (lambda: mk.grad_norm([table]), [], [table])):
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert [t._version for t in written] == [v + 1 for v in before[0]]
        assert [t._version for t in read] == before[1]
    w = torch.ones(12, device="cuda", requires_grad=True)
    y = (w * table).sum()
    mk.clip_grad_norm([table], 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        free = torch.ones((3, 12), device="cuda")
    mk.embedding(table, idx, out=free)                                    # has no version
    assert torch.equal(free, table[idx])


# ---------------------------------------------------------------- sorts of many tokens

# tiles of 8192 tokens and, from 152 of them on, several a CTA; one to three passes
@pytest.mark.parametrize("n,rows,width,skew", [(700001, 900, 4, 1), (700001, 30000, 3, 3), (1300003, 700, 3, 1),
                                               (1300003, 40000, 4, 2), (1300003, 1 << 21, 2, 1), (2500000, 1, 1, 1)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gradient_of_many_tokens(n, rows, width, skew, dtype):
    gen = generator(n + rows)
    idx = tokens(gen, n, rows, skew, torch.int64 if rows == 900 else torch.int32)
    grad = whole(gen, (n, width), TYPES[dtype])
    got = mk.embedding_grad(idx, grad, rows)
    assert torch.equal(got.double(), sums_in_64_bits(idx, grad, rows))
    acc = whole(gen, (rows, width), torch.float32)
    want = acc.double() + got.double()
    mk.embedding_grad(idx, grad, rows, out=acc, accumulate=True)
    assert torch.equal(acc.double(), want)


def model_in_64_bits(A, c, g=None):
    """Entries, and the gradients of all factors for g."""
    dims = torch.tensor([len(a) for a in A], device="cuda")
    c = c.long()
    inside = ((c >= 0) & (c < dims)).all(1)
    at = torch.where(inside[:, None], c, 0)
    rows = [a.double()[at[:, n]] * inside[:, None] for n, a in enumerate(A)]
    if g is None:
        return torch.stack(rows).prod(0).sum(1)
    grads = []
    for n, a in enumerate(A):
        term = (g.double() * inside)[:, None].expand(-1, a.shape[1]).clone()
        for m, r in enumerate(rows):
            if m != n:
                term *= r
        grads.append(torch.zeros_like(a, dtype=torch.float64).index_add_(0, at[:, n], term))
    return grads


def signs(gen, shape, dtype):
    return whole(gen, shape, dtype, 0, 2) * 2 - 1


# tiles of 8192 samples and several a CTA, by tables and (the last two) from the caches
@pytest.mark.parametrize("dims,R,S", [((64, 50, 40), 8, 262145), ((30,) * 6, 8, 204803), ((5,) * 8, 8, 160001),
                                      ((64, 50, 40), 12, 420001), ((9,), 5, 1300001),
                                      ((7000, 5000, 4000), 4, 262145), ((7000, 5000, 4000), 3, 420001)])
def test_entries_of_many_samples(dims, R, S):
    gen = generator(sum(dims) + S)
    A = [signs(gen, (n, R), torch.float32) for n in dims]
    c = torch.stack([tokens(gen, S, n) for n in dims], 1)
    g = whole(gen, (S,), torch.float32)
    assert torch.equal(mk.cp_entries(A, c).double(), model_in_64_bits(A, c))
    for n, (got, want) in enumerate(zip(mk.cp_entries_grad(A, c, g), model_in_64_bits(A, c, g))):
        assert torch.equal(got.double(), want), n


# ---------------------------------------------------------------- large results of few tokens

# results of more than 128 MB: zeros by many CTAs while a cluster sorts (a tile of 4096 tokens
# a CTA), also where the bytes are no multiple of 16; smaller ones, and at an odd offset, the
# rows have owners, or where they are too many the tokens are sorted by the whole GPU
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rows,width,dtype", [(200003, 127, "float32"), (400001, 127, "float16"), (200000, 128, "float32"),
                                              (800001, 65, "bfloat16"), (2000000, 16, "float32"),
                                              (270001, 127, "float32"), (540001, 127, "float16"), (270000, 128, "float32"),
                                              (1100001, 65, "bfloat16"), (2200000, 16, "float32")])
@pytest.mark.parametrize("n,skew", [(5000, 3), (16384, 1), (16384, 40), (16383, 2), (4097, 1)])
def test_gradient_of_few_tokens_into_a_large_table(n, skew, rows, width, dtype, offset):
    gen = generator(n + rows)
    idx = tokens(gen, n, rows, skew)
    grad = whole(gen, (n, width), TYPES[dtype], -1, 2)
    out, flat = placed(lambda k: torch.full((k,), 7.0, device="cuda", dtype=TYPES[dtype]), (rows, width), offset)
    mk.embedding_grad(idx, grad, rows, out=out)
    want = torch.zeros((rows, width), device="cuda")
    kept = ((idx >= 0) & (idx < rows)).nonzero().flatten()
    want.index_add_(0, idx[kept].long(), grad[kept].float())
    want = want.to(out.dtype)           # whole numbers: exact before this rounding
    assert torch.equal(out, want)
    assert torch.all(flat[:offset] == 7.0) and torch.all(flat[offset + rows * width:] == 7.0)


# ---------------------------------------------------------------- CP operands at odd offsets

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dims,R,S", [((12, 9, 15), 8, 500), ((300, 2, 50), 64, 5000), ((40, 30, 20), 36, 30000),
                                      ((20,) * 6, 32, 20000), ((48,) * 6, 16, 20000), ((9000, 4000), 16, 20000)])
@pytest.mark.parametrize("at,to", [(0, 1), (1, 0), (2, 3), (4, 2), (3, 4)])
def test_cp_operands_at_any_offset(dims, R, S, dtype, at, to):
    """Factors and results that start off 16 bytes, not all alike; what lies around results stays."""
    gen = generator(sum(dims) + S)
    A = [placed(lambda k: signs(gen, (k,), TYPES[dtype]), (n, R), at + m)[0] for m, n in enumerate(dims)]
    c = torch.stack([tokens(gen, S, n) for n in dims], 1)
    g, _ = placed(lambda k: whole(gen, (k,), torch.float32), (S,), at)
    x, room = placed(lambda k: torch.full((k,), 7.0, device="cuda"), (S,), to)
    assert mk.cp_entries(A, c, out=x) is x
    assert torch.equal(x.double(), model_in_64_bits(A, c))
    assert torch.all(room[:to] == 7.0) and torch.all(room[to + S:] == 7.0)
    outs, rooms = zip(*[placed(lambda k: torch.full((k,), 7.0, device="cuda"), (n, R), to) for n in dims])
    got = mk.cp_entries_grad(A, c, g, outs=list(outs))
    for out, room, n, mine, want in zip(outs, rooms, dims, got, model_in_64_bits(A, c, g)):
        assert mine.data_ptr() == out.data_ptr() and torch.equal(out.double(), want)
        assert torch.all(room[:to] == 7.0) and torch.all(room[to + n * R:] == 7.0)
