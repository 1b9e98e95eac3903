"""GPU rotation of rows by their position against the fp64 oracle on the same inputs.

Bound, with U = 2^-24 the unit roundoff of fp32: the angle within a quarter turn is rounded
by at most pi/4 U, what the fixed point leaves out is below 1e-8, sincospi is within one step
(2 U), the product with the scale adds U: a cosine or sine is within 4 U of scale; the two
products and their sum add 2 U of their magnitudes.  So |y - y'| <= 6 U scale (|u| + |v|) and
the result's rounding: v of its magnitude, or half the smallest step of its type."""
import numpy as np
import pytest

from oracle import orthogonal as oo

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
UNIT = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEP = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def f64(t):
    return t.double().cpu().numpy()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def check(x, positions, f, got, interleaved, scale=1.0, inverse=False):
    """x and got with a heads dimension."""
    n = len(f)
    want = oo.rotary(f64(x), positions.cpu().numpy(), f.numpy(), interleaved, scale, inverse)
    mag = np.abs(f64(x)[..., :2 * n])
    if interleaved:
        both = np.repeat(mag[..., 0::2] + mag[..., 1::2], 2, axis=-1)
    else:
        both = np.tile(mag[..., :n] + mag[..., n:], 2)
    bound = 6 * U * abs(scale) * both + UNIT[x.dtype] * np.abs(want[..., :2 * n]) * 1.01 + STEP[x.dtype]
    err = np.abs(f64(got)[..., :2 * n] - want[..., :2 * n])
    assert np.all(err <= bound), (err / bound).max()
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])


SHAPES = [  # batch, length, heads, width, dims
    (1, 1, 1, 2, 2), (1, 1, 32, 128, 128), (8, 1, 5, 128, 128), (2, 3, 7, 96, 64), (3, 33, 1, 17, 16), (1, 257, 3, 24, 24),
    (2, 129, 9, 12, 6), (1, 50, 2, 1030, 1024), (1, 40, 2, 300, 258), (2, 1001, 4, 80, 80), (1, 3000, 40, 64, 64),
    (1, 70000, 1, 10, 10), (5, 17, 13, 171, 168)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("batch,length,heads,width,dims", SHAPES)
def test_rotation(batch, length, heads, width, dims, interleaved, dtype):
    gen = generator(batch + length + width)
    x = normal(gen, (batch, length, heads, width), TYPES[dtype])
    f = mk.rotary_frequencies(dims)
    p = torch.randint(-1000, 1 << 20, (batch, length), generator=gen, device="cuda")
    p = p.int() if length % 2 else p
    got = mk.rotary(x, p, f, interleaved, scale=1.25)
    assert got.shape == x.shape and got.dtype == x.dtype
    check(x, p, f, got, interleaved, 1.25)
    back = mk.rotary_grad(x, p, f, interleaved, scale=0.5)
    check(x, p, f, back, interleaved, 0.5, inverse=True)
    same = x.clone()
    version = same._version
    assert mk.rotary(same, p, f, interleaved, scale=1.25, outs=same).data_ptr() == same.data_ptr()
    assert torch.equal(same, got) and same._version > version


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_extreme_positions(interleaved):
    """Whole turns and far positions: the angle is exact modulo a turn."""
    gen = generator(1)
    f = torch.tensor([1.0, -0.37, 1e-5, 2 * np.pi, 7.5, 1e-12], dtype=torch.float64)
    p = torch.tensor([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), (1 << 40) + 12345], device="cuda")
    x = normal(gen, (7, 2, 13), torch.float32)
    got = mk.rotary(x, p, f, interleaved)
    assert torch.equal(got[0], x[0])
    # a frequency's rounding to 53 bits moves the angle by p f 2^-53: it is part of the frequency,
    # but f / 2 pi is rounded once more, 2^-52 p f / 2 pi turns; up to 2^40 positions 1e-3 radians
    check(x[:4], p[:4], f, got[:4], interleaved)
    for t in (4, 5):
        want = oo.rotary(f64(x[t]), p[t].cpu().numpy(), f.numpy(), interleaved)
        assert np.abs(f64(got[t]) - want).max() < 1e-5
    assert torch.isfinite(got).all()


def test_layouts():
    """Shapes without heads or batch, shared positions, heads outside of tokens, rows at odd
    offsets, tensors of one buffer, expanded inputs."""
    gen = generator(2)
    f = mk.rotary_frequencies(16)
    base = normal(gen, (3, 20, 6, 16), torch.float32)
    p = torch.randint(0, 5000, (3, 20), generator=gen, device="cuda")
    want = mk.rotary(base, p, f)
    check(base, p, f, want, False)
    # rows: batch x length x width, length x width, length x heads x width
    assert torch.equal(mk.rotary(base[:, :, 2], p, f), want[:, :, 2])
    assert torch.equal(mk.rotary(base[1, :, 2], p[1], f), want[1, :, 2])
    assert torch.equal(mk.rotary(base[1], p[1], f), want[1])
    # positions shared by the batch, as one dimension, a batch of one, strides of zero; strided positions
    shared = mk.rotary(base, p[0], f)
    check(base, p[:1].expand(3, 20), f, shared, False)
    for q in (p[:1], p[:1].expand(3, 20), p[0].int(), torch.stack([p[0], p[1]], 1)[:, 0]):
        assert torch.equal(mk.rotary(base, q, f), shared)
    # heads outside of the tokens: the result keeps the layout
    outside = base.transpose(1, 2).contiguous().transpose(1, 2)
    got = mk.rotary(outside, p, f)
    assert torch.equal(got, want) and got.stride() == outside.stride()
    # parts of one buffer, in place, rows at an odd offset
    room = torch.zeros(3, 20, 6 * 16 + 6 * 16 + 3, device="cuda")
    a, b = room[:, :, 1:97].unflatten(2, (6, 16)), room[:, :, 98:194].unflatten(2, (6, 16))
    a.copy_(base)
    b.copy_(2.0 * base)
    ga, gb = mk.rotary([a, b], p, f, outs=[a, b])
    assert ga.data_ptr() == a.data_ptr() and torch.equal(a, want) and torch.equal(b, 2.0 * want)
    assert room[:, :, 0].abs().sum() == 0 and room[:, :, 97].abs().sum() == 0 and room[:, :, 194].abs().sum() == 0
    # into a given tensor, out of an expanded one
    out = torch.empty_like(base)
    one = base[:, :, :1].expand(3, 20, 6, 16)
    assert torch.equal(mk.rotary(one, p, f, outs=out), want[:, :, :1].expand(3, 20, 6, 16))
    assert torch.equal(mk.rotary(one, p, f), out)
    # several tensors of different numbers of heads in one call, one of none
    many = [base, base[:, :, :1], base[:, :, :0], base[:, :, 3:5]]
    for x, y in zip(many, mk.rotary(many, p, f)):
        assert torch.equal(y, mk.rotary(x, p, f) if x.numel() else x)
    assert mk.rotary(base[:0], p[:0], f).shape == (0, 20, 6, 16)
    assert mk.rotary(base[:, :0], p[:, :0], f).shape == (3, 0, 6, 16)


def test_results_of_many_heads():
    """More heads than the grid's second dimension holds."""
    gen = generator(3)
    f = mk.rotary_frequencies(2)
    x = normal(gen, (1, 70001, 2), torch.float32)
    p = torch.tensor([12345], device="cuda")
    check(x, p, f, mk.rotary(x, p, f), False)


def test_refusals():
    f = mk.rotary_frequencies(8)
    x, p = torch.zeros(4, 2, 8, device="cuda"), torch.arange(4, device="cuda")
    for kind, bad in [
            (TypeError, lambda: mk.rotary(x.double(), p, f)), (TypeError, lambda: mk.rotary(x, p.float(), f)),
            (TypeError, lambda: mk.rotary(x, p, f.cuda())), (TypeError, lambda: mk.rotary(x, p, f.float())),
            (TypeError, lambda: mk.rotary(x, p.cpu(), f)), (TypeError, lambda: mk.rotary(x, p, [1.0])),
            (ValueError, lambda: mk.rotary([], p, f)), (ValueError, lambda: mk.rotary([x] * 9, p, f)),
            (ValueError, lambda: mk.rotary(x, p[:3], f)), (ValueError, lambda: mk.rotary(x, p[None, None], f)),
            (ValueError, lambda: mk.rotary(x[..., 0], p[None], f)), (ValueError, lambda: mk.rotary(x.mT, p, f)),
            (ValueError, lambda: mk.rotary([x, x.half()], p, f)), (ValueError, lambda: mk.rotary([x, x[:2]], p, f)),
            (ValueError, lambda: mk.rotary(x, p, f, outs=x[:, :1])), (ValueError, lambda: mk.rotary([x], p, f, outs=[])),
            (mk.MttkrpError, lambda: mk.rotary(x, p, mk.rotary_frequencies(10))),
            (mk.MttkrpError, lambda: mk.rotary([x, x], p, f, outs=[x, x])),
            (mk.MttkrpError, lambda: mk.rotary(x, p, f, outs=x[:1].expand(4, 2, 8)))]:
        with pytest.raises(kind):
            bad()
    assert x.abs().sum() == 0


def test_streams_and_graphs():
    gen = generator(4)
    f = mk.rotary_frequencies(64)
    x = normal(gen, (2, 300, 8, 64), torch.bfloat16)
    p = torch.randint(0, 1 << 17, (2, 300), generator=gen, device="cuda")
    want = mk.rotary(x, p, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mk.rotary(x, p, f, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mk.rotary(x, p, f, outs=out)
    y = normal(gen, (2, 300, 8, 64), torch.bfloat16)
    x.copy_(y)
    p.add_(77)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mk.rotary(y, p, f))


def test_positions_and_infinities():
    """What is not finite stays with its pair; the columns that are copied keep their bits."""
    f = mk.rotary_frequencies(4)
    x = torch.ones(3, 1, 6, device="cuda")
    x[1, 0, 0] = float("inf")
    x[1, 0, 5] = float("nan")
    got = mk.rotary(x, torch.tensor([5, 6, 7], device="cuda"), f)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all()
    assert not torch.isfinite(got[1, 0, [0, 2]]).any() and torch.isfinite(got[1, 0, [1, 3, 4]]).all()
    assert torch.isnan(got[1, 0, 5])


def test_positions_give_lookups_their_turn():
    """Lookup, rotation, and back: the gradient of a table through both."""
    gen = generator(5)
    table = normal(gen, (50, 24), torch.float32)
    idx = torch.randint(-1, 50, (200,), generator=gen, device="cuda")
    p = torch.randint(0, 9999, (200,), generator=gen, device="cuda")
    f = mk.rotary_frequencies(16)
    rows = mk.rotary(mk.embedding(table, idx), p, f)
    g = normal(gen, (200, 24), torch.float32)
    grad = mk.embedding_grad(idx, mk.rotary_grad(g, p, f), 50)
    lhs = float((rows.double() * g.double()).sum())
    rhs = float((grad.double() * table.double()).sum())
    # both are sums of 200 x 24 products of normals: sqrt(4800) in size, each product within 16 U
    assert abs(lhs - rhs) <= 32 * U * float((rows.abs().double() * g.abs().double()).sum() * 2)


DENSE = [  # batch, length, heads of each tensor, width, dims: rows at odd offsets that follow one another
    (1, 1, (1,), 3, 2), (2, 3, (5, 1), 7, 6), (1, 700, (3,), 13, 12), (3, 1001, (1,), 9, 8), (2, 650, (8, 2), 83, 66),
    (1, 900, (4,), 1031, 1024), (1, 5, (47,), 1045, 1000), (1, 3, (48,), 1047, 10), (4, 7, (2, 30, 1), 171, 168)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("batch,length,heads,width,dims", DENSE)
def test_dense_rows_at_odd_offsets(batch, length, heads, width, dims, shift, interleaved, dtype):
    """Tensors that fill their memory, as tokens of heads and as heads of tokens, with what lies around
    them left as it was; the same values as from rows that do not follow one another."""
    gen = generator(length + width + shift)
    f = mk.rotary_frequencies(dims)
    p = torch.randint(-1000, 1 << 20, (batch, length), generator=gen, device="cuda")
    for outside in (False, True):
        xs, outs, rooms = [], [], []
        for h in heads:
            shape = (batch, h, length, width) if outside else (batch, length, h, width)
            n = batch * h * length * width
            rooms.append(torch.full((n + 17,), 7.0, device="cuda", dtype=TYPES[dtype]))
            x = torch.empty(n + 17, device="cuda", dtype=TYPES[dtype])[shift:shift + n].view(shape)
            x.copy_(normal(gen, shape, TYPES[dtype]))
            out = rooms[-1][shift:shift + n].view(shape)
            xs.append(x.transpose(1, 2) if outside else x)
            outs.append(out.transpose(1, 2) if outside else out)
        mk.rotary(xs, p, f, interleaved, scale=1.25, outs=outs)
        for x, out, room, h in zip(xs, outs, rooms, heads):
            check(x, p, f, out, interleaved, 1.25)
            n = batch * h * length * width
            assert (room[:shift] == 7).all() and (room[shift + n:] == 7).all()
            apart = torch.zeros(batch, length, h, width + 2, device="cuda", dtype=TYPES[dtype])
            apart[..., :width] = x
            assert torch.equal(mk.rotary(apart[..., :width], p, f, interleaved, scale=1.25), out)
        again = [x.clone(memory_format=torch.preserve_format) for x in xs]
        mk.rotary(again, p, f, interleaved, scale=1.25, outs=again)
        assert all(torch.equal(x, y) for x, y in zip(again, outs))
