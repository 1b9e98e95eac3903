"""What the orthogonal maps' C entry points and their binding refuse, on the host, before
anything is enqueued (every pointer below is made up and never dereferenced)."""
import ctypes

import pytest

import dense_tensor_decomposition_gb300 as mk

F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    mk.build()
    return mk.load_library()


def refused(lib, rc, why, code=1):
    assert rc == code, (rc, lib.mttkrp_last_error())
    assert why.lower() in lib.mttkrp_last_error().decode().lower()


class Tensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("x_strides", ctypes.c_int64 * 3), ("out_strides", ctypes.c_int64 * 3)]


def rows(x=0x100000, out=0x200000, heads=2, xs=(160, 32, 16), ys=(160, 32, 16)):
    return Tensor(x, out, heads, (ctypes.c_int64 * 3)(*xs), (ctypes.c_int64 * 3)(*ys))


def rotary(lib, tensors=(rows(),), n=None, type=F32, batch=3, length=5, width=16, positions=0x10000, pos_bytes=8,
           pos_strides=(0, 1), freqs=(1.0, 0.5, 0.25), dims=6, null=False):
    n = len(tensors) if n is None else n
    array = None if null else (Tensor * max(len(tensors), 1))(*tensors)
    f = (ctypes.c_double * 512)(*freqs) if freqs is not None else None
    return lib.mttkrp_rotary(n, array, type, batch, length, width, positions, pos_bytes, *pos_strides, f, dims, 0, 1.0,
                             0, None)


@pytest.mark.parametrize("change,why", [
    ({"n": 0}, "tensors outside"), ({"n": 9}, "tensors outside"), ({"null": True}, "NULL"), ({"freqs": None}, "NULL"),
    ({"type": 3}, "type"), ({"batch": -1}, "tokens"), ({"length": -1}, "tokens"), ({"batch": 1 << 16, "length": 1 << 15}, "tokens"),
    ({"width": 0}, "width"), ({"width": 65537}, "width"), ({"dims": 5}, "dims"), ({"dims": 0}, "dims"),
    ({"dims": 18}, "dims"), ({"dims": 1026, "width": 4000}, "dims"), ({"pos_bytes": 2}, "bytes"),
    ({"positions": 0}, "positions"), ({"positions": 0x10004}, "aligned"), ({"pos_strides": (0, -1)}, "negative"),
    ({"pos_strides": (1 << 40, 1)}, "2^40"),
    ({"freqs": (1.0, float("inf"), 0.0)}, "frequency 1"), ({"freqs": (1.0, float("nan"), 0.0)}, "frequency 1")])
def test_rotation_refuses(lib, change, why):
    refused(lib, rotary(lib, **change), why)


@pytest.mark.parametrize("tensors,why", [
    ([rows(heads=-1)], "heads"), ([rows(x=0)], "NULL"), ([rows(out=0)], "NULL"), ([rows(x=0x100002)], "aligned"),
    ([rows(xs=(-1, 32, 16))], "negative"), ([rows(ys=(160, -32, 16))], "negative"), ([rows(xs=(1 << 40, 32, 16))], "2^40"),
    ([rows(ys=(160, 32, 15))], "rows overlap"), ([rows(ys=(0, 32, 16))], "rows overlap"),
    ([rows(ys=(160, 31, 16))], "rows overlap"), ([rows(out=0x100004)], "without being it"),
    ([rows(out=0x100000, ys=(200, 40, 16))], "without being it"), ([rows(out=0x10000 - 16)], "positions"),
    ([rows(), rows()], "overlap"), ([rows(), rows(x=0x300000, out=0x200010)], "overlap"),
    ([rows(), rows(x=0x300000, out=0x100000)], "overlaps tensor"),
    ([rows(out=0x100000), rows(x=0x100000)], "overlaps tensor"),
    ([rows(out=0x100000), rows(x=0x100000 + 64, out=0x300000)], "overlaps tensor")])
def test_rotation_refuses_tensors(lib, tensors, why):
    refused(lib, rotary(lib, tensors=tensors), why)


def no_launch(lib, tensors, **more):
    """Everything is taken up to the launch, which a machine without a GPU refuses."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are not for a GPU")
    assert rotary(lib, tensors=tensors, **more) == 4, lib.mttkrp_last_error()


def test_rotation_takes_parts_of_one_buffer(lib):
    """In place, queries and keys beside one another in every token (and in every sequence
    where heads lie outside the tokens): their spans overlap, their rows do not."""
    token = 4 * 16                      # 2 heads of each of two tensors
    for first in (0, 1):
        both = [rows(x=0x100000 + 128 * k, out=0x100000 + 128 * k, xs=(5 * token, token, 16), ys=(5 * token, token, 16))
                for k in (first, 1 - first)]
        no_launch(lib, both)
        outside = [rows(x=0x100000 + 2 * 5 * 64 * k, out=0x100000 + 2 * 5 * 64 * k, xs=(4 * 5 * 16, 16, 5 * 16),
                        ys=(4 * 5 * 16, 16, 5 * 16)) for k in (first, 1 - first)]
        no_launch(lib, outside)
    refused(lib, rotary(lib, tensors=[rows(x=0x100000, out=0x100000, xs=(5 * token, token, 16), ys=(5 * token, token, 16)),
                                      rows(x=0x100000 + 64, out=0x100000 + 64, xs=(5 * token, token, 16),
                                           ys=(5 * token, token, 16))]), "overlap")


def test_rotation_of_nothing_is_done(lib):
    assert rotary(lib, batch=0) == 0 and rotary(lib, length=0, positions=0) == 0
    assert rotary(lib, tensors=[rows(heads=0, x=0, out=0)]) == 0


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x, p, f = torch.zeros(4, 2, 8), torch.arange(4), mk.rotary_frequencies(8)
    for bad in (lambda: mk.rotary(x, p, f), lambda: mk.rotary_grad([x], p, f)):
        with pytest.raises(TypeError):
            bad()


class Matrices(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("type", ctypes.c_int)]


def matrix(data=0x1000000, batch=2, rows=6, cols=5, batch_stride=40, row_stride=6, type=F32):
    return Matrices(data, batch, rows, cols, batch_stride, row_stride, type)


def listed(ms):
    return None if ms is None else (Matrices * max(len(ms), 1))(*ms)


QUINTIC = (3.4445, -4.775, 2.0315)


def orthogonalize(lib, ins=(matrix(),), outs=(matrix(0x2000000),), n=None, steps=5, abc=QUINTIC * 5, eps=1e-7,
                  scales=None, ws=0x4000000, ws_bytes=1 << 30):
    n = len(ins) if n is None else n
    c = None if abc is None else (ctypes.c_double * max(len(abc), 3))(*abc)
    return lib.mttkrp_orthogonalize(n, listed(ins), listed(outs), steps, c, eps, scales, ws, ws_bytes, None)


HERE = 0x1000000
# a matrix of which no side is short: it needs a workspace
BIG_SHAPE = dict(batch=1, rows=130, cols=200, batch_stride=0, row_stride=200)
LARGE = dict(ins=[matrix(HERE, **BIG_SHAPE)], outs=[matrix(0x2000000, **BIG_SHAPE)])


@pytest.mark.parametrize("change,why,code", [
    ({"n": -1}, "n=", 1), ({"n": (1 << 20) + 1}, "n=", 1), ({"ins": None, "n": 1}, "NULL", 1), ({"outs": None}, "NULL", 1),
    ({"ins": [matrix(rows=-1)]}, "range", 1), ({"ins": [matrix(cols=1 << 19)]}, "range", 1),
    ({"ins": [matrix(batch=1 << 31)]}, "range", 1), ({"ins": [matrix(rows=1 << 18, cols=1 << 18)]}, "128 GB", 1),
    ({"ins": [matrix(type=7)]}, "type", 1), ({"outs": [matrix(0x2000000, type=-1)]}, "type", 1),
    ({"ins": [matrix(0)]}, "NULL", 1), ({"outs": [matrix(0)]}, "NULL", 1), ({"ins": [matrix(HERE + 2)]}, "aligned", 1),
    ({"ins": [matrix(row_stride=4)]}, "closer", 1), ({"ins": [matrix(batch_stride=34)]}, "overlap", 1),
    ({"ins": [matrix(row_stride=-6)]}, "negative", 1), ({"ins": [matrix(row_stride=1 << 40)]}, "2^40", 1),
    ({"outs": [matrix(0x2000000, rows=5)]}, "shape", 1), ({"outs": [matrix(0x2000000, batch=1)]}, "shape", 1),
    ({"outs": [matrix(HERE + 4)]}, "overlaps", 1), ({"outs": [matrix(HERE, row_stride=7)]}, "overlaps", 1),
    ({"outs": [matrix(HERE, type=BF16, row_stride=6)]}, "overlaps", 1),
    ({"ins": [matrix(), matrix(0x3000000)], "outs": [matrix(0x2000000), matrix(0x2000010)]}, "overlaps", 1),
    ({"ins": [matrix(), matrix(0x3000000)], "outs": [matrix(0x2000000), matrix(HERE)]}, "overlaps", 1),
    ({"ins": [matrix(), matrix()], "outs": [matrix(HERE), matrix(0x2000000)]}, "overlaps", 1),
    ({"steps": 0}, "steps", 1), ({"steps": 65}, "steps", 1), ({"abc": None}, "NULL", 1), ({"eps": -1.0}, "eps", 1),
    ({"eps": float("nan")}, "eps", 1), ({"eps": float("inf")}, "eps", 1),
    ({"abc": QUINTIC * 4 + (float("nan"), 0, 0)}, "finite", 1), ({"abc": (16.0, 0, 0) * 5}, "15.9", 1),
    ({"abc": (2.0, 0, 0) * 5}, "3.9", 1), ({"abc": (4.0, 0, 0) + QUINTIC * 4}, "3.9", 1),
    ({"abc": (1.0, 14.95, -13.0) + QUINTIC * 4}, "3.9", 1),     # 4.26 at s^2 = 0.79 (-14 reaches 3.87: taken)
    ({**LARGE, "ws": 0}, "workspace", 3), ({**LARGE, "ws_bytes": 100}, "workspace", 3),
    ({**LARGE, "ws": 0x4000080}, "256-byte", 3)])
def test_orthogonalisation_refuses(lib, change, why, code):
    refused(lib, orthogonalize(lib, **change), why, code)


def test_orthogonalisation_takes_what_fits(lib):
    """Up to the status word, which a machine without a GPU does not have: in place, columns of
    one buffer, coefficients whose last step grows, no matrices."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are not for a GPU")
    assert orthogonalize(lib, outs=[matrix(HERE)]) == 4
    left, right = matrix(HERE, 1, 6, 5, 0, 12), matrix(HERE + 24, 1, 6, 5, 0, 12)
    assert orthogonalize(lib, ins=[left, right], outs=[left, right]) == 4
    assert orthogonalize(lib, ins=[right, left], outs=[right, left]) == 4
    refused(lib, orthogonalize(lib, ins=[left, right], outs=[right, left]), "overlaps")
    assert orthogonalize(lib, steps=1, abc=(15.0, 0.0, 0.0)) == 4
    assert orthogonalize(lib, ins=[], outs=[]) == 0
    assert orthogonalize(lib, ins=[matrix(0, rows=0)], outs=[matrix(0, rows=0)], ws=0, ws_bytes=0) == 0


def test_orthogonalisation_workspace(lib):
    size = lambda *ms: lib.mttkrp_orthogonalize_workspace_bytes(len(ms), listed(ms))
    one = size(matrix(batch=1, rows=192, cols=192, batch_stride=0, row_stride=192))
    assert 72 * 8192 <= one < 72 * 8192 + 4096
    assert size(matrix(batch=3, rows=200, cols=500, row_stride=500, batch_stride=100000)) >= 3 * 4 * (4 * 8 + 16) * 8192
    assert size(matrix(batch=3, rows=100, cols=1500, row_stride=1500, batch_stride=150000)) == 0      # one launch, no workspace
    assert size(matrix(batch=1, rows=100, cols=1600, batch_stride=0, row_stride=1600)) > 0            # beyond a cluster
    assert size(matrix(batch=1, rows=7000, cols=64, batch_stride=0, row_stride=64)) > 0
    # a list beyond 4 GB goes in parts
    big = matrix(batch=100, rows=4096, cols=4096, row_stride=4096, batch_stride=1 << 24)
    assert size(big) <= (4 << 30) + (1 << 20) and size(big, big) <= (4 << 30) + (1 << 20)
    assert size(matrix(rows=-1)) == 0 and size(matrix(batch=0)) == 0 and lib.mttkrp_orthogonalize_workspace_bytes(0, None) == 0


def step(lib, weights=None, grads=None, momenta=None, weights_out=None, momenta_out=None, lr=0.1, momentum=0.9, wd=0.0,
         steps=5, ws=0x40000000):
    at = lambda k, ms: listed(ms if ms is not None else [matrix(0x1000000 * (k + 1))])
    c = (ctypes.c_double * 15)(*(QUINTIC * 5))
    return lib.mttkrp_orthogonal_step(1, at(0, weights), at(1, grads), at(2, momenta), at(3, weights_out), at(4, momenta_out),
                                      lr, momentum, 1, wd, steps, c, 1e-7, None, ws, 1 << 30, None)


@pytest.mark.parametrize("change,why", [
    ({"weights": [matrix(rows=7, batch_stride=60)]}, "shape"), ({"momenta": [matrix(0)]}, "NULL"),
    ({"weights_out": [matrix(0x4000000, type=BF16)]}, "type"), ({"momenta_out": [matrix(0x5000000, type=F16)]}, "type"),
    ({"weights_out": [matrix(0x2000000)]}, "overlaps"), ({"momenta_out": [matrix(0x1000000)]}, "overlaps"),
    ({"momenta_out": [matrix(0x4000000)]}, "overlaps"), ({"weights_out": [matrix(0x1000004)]}, "overlaps"),
    ({"lr": float("nan")}, "finite"), ({"momentum": float("inf")}, "finite"), ({"wd": float("nan")}, "finite"),
    ({"steps": 0}, "steps")])
def test_step_refuses(lib, change, why):
    refused(lib, step(lib, **change), why)
