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
