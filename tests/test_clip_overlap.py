"""Clipping refuses results that overlap one another or another tensor, on the host, before
anything is enqueued (every pointer below is made up and never dereferenced; what passes
ends at the missing workspace)."""
import ctypes
import random

import pytest

import dense_tensor_decomposition_gb300 as mk

F32, BF16 = 0, 1
INVALID, WORKSPACE = 1, 3
BYTES = {F32: 4, BF16: 2}


@pytest.fixture(scope="module")
def lib():
    mk.build()
    return mk.load_library()


def clip(lib, tensors, numels, types, outs=None):
    n = len(tensors)
    co = (ctypes.c_void_p * n)(*outs) if outs is not None else None
    return lib.mttkrp_clip_grad_norm(n, (ctypes.c_void_p * n)(*tensors), (ctypes.c_int64 * n)(*numels),
                                     (ctypes.c_int * n)(*types), co, 1.0, 1e-6, 0x1000, None, 0, None)


A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000


@pytest.mark.parametrize("tensors,numels,outs", [
    ((A, A), (10, 10), None),                               # the same tensor twice, in place
    ((B, A, B), (10, 7, 10), None),
    ((A, A + 36), (10, 10), None),                          # its last element
    ((A + 36, A), (10, 10), None),
    ((A, A + 400), (1000, 10), None),                       # a part of it
    ((A, B), (10, 10), (C, C)),                             # one result for two
    ((A, B), (10, 10), (C + 36, C)),
    ((A, B), (10, 10), (B, C)),                             # the other one's input
    ((A, B), (10, 10), (C, A + 4)),
    ((A, B), (10, 10), (B, A)),
    ((A, B, C), (10, 1000, 10), (A, D, B + 2000)),
    ((A, A), (10, 10), (A, C)),
    (tuple(A + 64 * k for k in range(3000)) + (A + 64 * 1234,), (16,) * 3001, None)])
def test_refused(lib, tensors, numels, outs):
    assert clip(lib, tensors, numels, (F32,) * len(tensors), outs) == INVALID
    assert "overlap" in lib.mttkrp_last_error().decode()


@pytest.mark.parametrize("tensors,numels,outs", [
    ((A, B), (10, 10), None), ((B, A), (10, 10), None),
    ((A, A + 40), (10, 10), None), ((A + 40, A), (10, 10), None),               # neighbours
    ((A, A), (10, 10), (C, D)),                                                 # read twice
    ((A, A + 20), (10, 10), (C, D)),
    ((A, B), (10, 10), (A, C)), ((A, B), (10, 10), (C, B)),                     # one in place
    ((A, A, B), (10, 0, 10), None), ((A, B, B), (10, 10, 10), (C, D, D + 40)),
    (tuple(A + 64 * (k * 7 % 3000) for k in range(3000)), (16,) * 3000, None)])
def test_taken(lib, tensors, numels, outs):
    assert clip(lib, tensors, numels, (F32,) * len(tensors), outs) == WORKSPACE


def test_like_a_look_at_all_pairs(lib):
    rng = random.Random(4)
    seen = set()
    for _ in range(4000):
        n = rng.randint(1, 6)
        numels = [rng.choice([0, 1, 2, 5, 9]) for _ in range(n)]
        types = [rng.choice([F32, BF16]) for _ in range(n)]
        # even addresses of a few hundred bytes, at their type's alignment
        at = [[A + BYTES[t] * rng.randrange(160 // BYTES[t]) for t in types] for _ in range(2)]
        outs = [x if rng.random() < 0.5 else y for x, y in zip(*at)] if rng.random() < 0.7 else None
        to = at[0] if outs is None else outs
        spans = [[(x, x + k * BYTES[t]) for x, k, t in zip(w, numels, types)] for w in (at[0], to)]

        def meet(a, b):
            return a[0] < a[1] and b[0] < b[1] and a[0] < b[1] and b[0] < a[1]

        bad = any(meet(spans[1][i], spans[1][j]) for i in range(n) for j in range(i))
        bad |= any(meet(spans[1][i], spans[0][j]) and (i != j or to[i] != at[0][j]) for i in range(n) for j in range(n))
        assert clip(lib, at[0], numels, types, outs) == (INVALID if bad else WORKSPACE), (at, numels, types, outs)
        seen.add((bad, outs is None))
    assert len(seen) == 4
