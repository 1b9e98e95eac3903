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
