"""Lists of the orthogonal maps that are one array, as a C caller may pass them: what overlaps is refused
just as with equal arrays (every pointer below is made up and never dereferenced)."""
import ctypes

import pytest

import dense_tensor_decomposition_gb300 as mk


class Matrices(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("type", ctypes.c_int)]


W, G, M, A, B = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000


@pytest.fixture(scope="module")
def lib():
    mk.build()
    return mk.load_library()


@pytest.fixture(autouse=True)
def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up pointers are not for a GPU")


def step(lib, *at):
    """weights, gradients, momenta, new weights, new momenta at these addresses: as one array where the
    address is the same, and as arrays of their own; the two results, which have to agree."""
    abc = (ctypes.c_double * 15)(*((3.4445, -4.775, 2.0315) * 5))
    own = [(Matrices * 1)(Matrices(a, 2, 6, 5, 40, 6, 0)) for a in at]
    shared = [next(x for x, b in zip(own, at) if b == a) for a in at]
    codes = [lib.mttkrp_orthogonal_step(1, *lists, 0.1, 0.9, 1, 0.0, 5, abc, 1e-7, None, None, 0, None)
             for lists in (own, shared)]
    assert codes[0] == codes[1], at
    return codes[0]


def test_a_step(lib):
    taken = 4                               # up to the status word, which a machine without a GPU does not have
    assert step(lib, W, G, M, A, B) == taken and step(lib, W, G, M, W, M) == taken
    assert step(lib, W, G, M, W, B) == taken and step(lib, W, W, W, A, B) == taken
    for at in ((W, W, M, W, B), (W, W, W, W, W), (W, G, W, W, B), (W, G, W, W, W), (W, G, M, G, B), (W, G, M, M, B),
               (W, G, M, A, W), (W, G, M, A, G), (W, G, G, A, G), (W, G, M, A, A)):
        assert step(lib, *at) == 1 and b"overlaps" in lib.mttkrp_last_error(), at


def test_orthogonalisation(lib):
    abc = (ctypes.c_double * 15)(*((3.4445, -4.775, 2.0315) * 5))
    two = (Matrices * 2)(Matrices(W, 2, 6, 5, 40, 6, 0), Matrices(G, 2, 6, 5, 40, 6, 0))
    assert lib.mttkrp_orthogonalize(2, two, two, 5, abc, 1e-7, None, None, 0, None) == 4
    same = (Matrices * 2)(two[0], two[0])
    assert lib.mttkrp_orthogonalize(2, same, same, 5, abc, 1e-7, None, None, 0, None) == 1
