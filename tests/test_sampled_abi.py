"""What the sampled operators' C entry points refuse, on the host, before anything is
enqueued (every pointer below is made up and never dereferenced)."""
import ctypes

import pytest

import dense_tensor_decomposition_gb300 as mk

F32, BF16, F16 = 0, 1, 2
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    mk.build()
    return mk.load_library()


def refused(lib, rc, why, code=1):
    assert rc == code
    assert why.lower() in lib.mttkrp_last_error().decode().lower()


LOOKUP = dict(table=0x100000, rows=100, width=8, table_stride=8, type=F32, idx=0x10000, n=16, idx_stride=1,
              idx_bytes=8, scale=1.0, out=0x200000, out_stride=8)


@pytest.mark.parametrize("change,why", [
    ({"rows": 0}, "rows"), ({"rows": 1 << 31}, "rows"), ({"width": 0}, "width"), ({"width": 65537, "table_stride": 1 << 20}, "width"),
    ({"table_stride": 7}, "closer"), ({"out_stride": 7}, "closer"), ({"type": 3}, "type"), ({"type": -1}, "type"),
    ({"idx": 0}, "indices"), ({"idx_bytes": 2}, "bytes"), ({"idx": 0x10004}, "aligned"), ({"idx_stride": -1}, "stride"),
    ({"n": -1}, "n="), ({"n": 1 << 31}, "n="), ({"table": 0}, "table"), ({"out": 0}, "result"),
    ({"table": 0x100002}, "aligned"), ({"out": 0x200001, "type": BF16}, "aligned"),
    ({"out": 0x100000}, "overlap"), ({"out": 0x100000 + 100 * 32 - 4}, "overlap"), ({"out": 0x10000 - 16 * 32 + 4}, "overlap"),
    ({"table_stride": BIG}, "2^40")])
def test_lookup_refuses(lib, change, why):
    refused(lib, lib.mttkrp_embedding(*{**LOOKUP, **change}.values(), None), why)


# tokens and samples enough for the gradients to need their workspace
GRAD = dict(idx=0x10000, n=20000, idx_stride=1, idx_bytes=4, grad=0x100000, type=BF16, grad_stride=8, rows=100, width=8,
            scale=1.0, accumulate=0, out=0x200000, out_type=F32, out_stride=8, ws=0x400000, ws_bytes=1 << 20)


@pytest.mark.parametrize("change,why,code", [
    ({"rows": 0}, "rows", 1), ({"rows": 1 << 31}, "rows", 1), ({"n": -1}, "n=", 1), ({"idx": 0}, "indices", 1),
    ({"idx": 0x10002}, "aligned", 1), ({"grad": 0}, "gradient", 1), ({"grad_stride": 4}, "closer", 1),
    ({"out_type": F16}, "fp32", 1), ({"out_type": 9}, "type", 1), ({"type": 9}, "type", 1), ({"out": 0}, "result", 1),
    ({"out": 0x200002}, "aligned", 1), ({"out": 0x100000 + 4}, "overlap", 1), ({"out": 0x10000 - 4}, "overlap", 1),
    ({"ws": 0}, "workspace", 3), ({"ws_bytes": 100}, "workspace", 3), ({"ws": 0x400080}, "256-byte", 3)])
def test_lookup_gradient_refuses(lib, change, why, code):
    refused(lib, lib.mttkrp_embedding_grad(*{**GRAD, **change}.values(), None), why, code)


def model(d=3, dims=(30, 20, 10), R=8, factors=(0x100000, 0x110000, 0x120000), type=F32, coords=0x10000, n=20000,
          idx_bytes=4):
    cd = (ctypes.c_int64 * len(dims))(*dims) if dims is not None else None
    cf = (ctypes.c_void_p * len(factors))(*factors) if factors is not None else None
    return d, cd, R, cf, type, coords, n, idx_bytes


BAD_MODELS = [({"d": 0}, "order"), ({"d": 9, "dims": (2,) * 9, "factors": (0x100000,) * 9}, "order"),
              ({"dims": None}, "NULL"), ({"factors": None}, "NULL"), ({"dims": (30, 0, 10)}, "dims[1]"),
              ({"dims": (30, 1 << 31, 10)}, "dims[1]"), ({"R": 0}, "rank"), ({"R": 70000}, "rank"),
              ({"factors": (0x100000, 0, 0x120000)}, "NULL"), ({"factors": (0x100000, 0x110002, 0x120000)}, "aligned"),
              ({"type": 5}, "type"), ({"coords": 0}, "indices"), ({"coords": 0x10002}, "aligned"),
              ({"idx_bytes": 3}, "bytes"), ({"n": 1 << 31}, "n=")]


@pytest.mark.parametrize("change,why", BAD_MODELS)
def test_entries_refuse(lib, change, why):
    refused(lib, lib.mttkrp_cp_entries(*model(**change), 0x300000, None), why)


@pytest.mark.parametrize("out,why", [(0, "result"), (0x300002, "aligned"), (0x110010, "overlap"), (0x10010, "overlap")])
def test_entries_refuse_results(lib, out, why):
    refused(lib, lib.mttkrp_cp_entries(*model(), out, None), why)


OUTS = (0x300000, 0x310000, 0x320000)


@pytest.mark.parametrize("change,why", BAD_MODELS)
def test_entries_gradient_refuses(lib, change, why):
    outs = (ctypes.c_void_p * 3)(*OUTS)
    refused(lib, lib.mttkrp_cp_entries_grad(*model(**change), 0x20000, outs, 0x400000, 1 << 20, None), why)


@pytest.mark.parametrize("outs,g,ws,ws_bytes,why,code", [
    (None, 0x20000, 0x400000, 1 << 20, "results", 1), (OUTS, 0, 0x400000, 1 << 20, "gradient", 1),
    ((0x300000, 0, 0x320000), 0x20000, 0x400000, 1 << 20, "NULL", 1),
    ((0x300000, 0x300010, 0x320000), 0x20000, 0x400000, 1 << 20, "overlap", 1),
    ((0x300000, 0x310000, 0x120010), 0x20000, 0x400000, 1 << 20, "overlap", 1),
    ((0x300000, 0x310000, 0x20010), 0x20000, 0x400000, 1 << 20, "overlap", 1),
    (OUTS, 0x20000, 0, 0, "workspace", 3), (OUTS, 0x20000, 0x400000, 64, "workspace", 3),
    (OUTS, 0x20000, 0x400010, 1 << 24, "256-byte", 3)])
def test_entries_gradient_refuses_results(lib, outs, g, ws, ws_bytes, why, code):
    co = (ctypes.c_void_p * 3)(*outs) if outs is not None else None
    refused(lib, lib.mttkrp_cp_entries_grad(*model(), g, co, ws, ws_bytes, None), why, code)


def clip(lib, tensors=(0x100000, 0x200000), numels=(10, 20), types=(F32, BF16), outs=None, max_norm=1.0, eps=1e-6,
         norm=0x1000, ws=0x400000, ws_bytes=1 << 20, n=None):
    n = len(tensors) if n is None else n
    co = (ctypes.c_void_p * n)(*outs) if outs is not None else None
    return lib.mttkrp_clip_grad_norm(n, (ctypes.c_void_p * n)(*tensors), (ctypes.c_int64 * n)(*numels),
                                     (ctypes.c_int * n)(*types), co, max_norm, eps, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("change,why,code", [
    ({"types": (F32, 7)}, "type", 1), ({"numels": (10, -1)}, "elements", 1), ({"numels": (BIG, 1)}, "2^40", 1),
    ({"tensors": (0, 0x200000)}, "tensor 0", 1), ({"tensors": (0x100002, 0x200000)}, "aligned", 1),
    ({"outs": (0x300000, 0)}, "result 1", 1), ({"outs": (0x300000, 0x300101)}, "result 1", 1),
    ({"outs": (0x100004, 0x300000)}, "overlaps", 1), ({"max_norm": -1.0}, "max_norm", 1),
    ({"max_norm": float("nan")}, "max_norm", 1), ({"eps": -1.0}, "eps", 1), ({"norm": 0}, "norm", 1),
    ({"norm": 0x1002}, "norm", 1), ({"ws": 0}, "workspace", 3), ({"ws_bytes": 8}, "workspace", 3),
    ({"ws": 0x400004}, "256-byte", 3)])
def test_clipping_refuses(lib, change, why, code):
    refused(lib, clip(lib, **change), why, code)


def test_clipping_refuses_bad_lists(lib):
    refused(lib, lib.mttkrp_clip_grad_norm(-1, None, None, None, None, 1.0, 0.0, 0x1000, 0x400000, 1 << 20, None), "n=")
    refused(lib, lib.mttkrp_grad_norm((1 << 20) + 1, None, None, None, 0x1000, 0x400000, 1 << 20, None), "n=")
    refused(lib, lib.mttkrp_grad_norm(2, None, None, None, 0x1000, 0x400000, 1 << 20, None), "NULL")


def test_workspace_sizes(lib):
    assert lib.mttkrp_embedding_grad_workspace_bytes(-1, 5, 5) == 0
    assert lib.mttkrp_embedding_grad_workspace_bytes(5, 0, 5) == 0
    dims = (ctypes.c_int64 * 3)(4, 5, 6)
    assert lib.mttkrp_embedding_grad_workspace_bytes(1000, 50, 64) == 0       # one launch, no workspace
    assert lib.mttkrp_embedding_grad_workspace_bytes(1000, 1 << 24, 64) >= 1000 * 8
    assert lib.mttkrp_embedding_grad_workspace_bytes(100000, 50, 64) >= 100000 * 8
    assert lib.mttkrp_cp_entries_grad_workspace_bytes(3, dims, 64, 1000) == 0
    assert lib.mttkrp_cp_entries_grad_workspace_bytes(3, dims, 64, 100000) >= 3 * 100000 * 16
    assert lib.mttkrp_cp_entries_grad_workspace_bytes(9, dims, 64, 1000) == 0
    assert lib.mttkrp_grad_norm_workspace_bytes(-1) == 0
    assert 0 < lib.mttkrp_grad_norm_workspace_bytes(1) < lib.mttkrp_grad_norm_workspace_bytes(1 << 20)


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    t, i = torch.zeros(4, 3), torch.zeros(2, dtype=torch.int64)
    for bad in (lambda: mk.embedding(t, i), lambda: mk.embedding_grad(i, t[:2], 4), lambda: mk.grad_norm([t]),
                lambda: mk.cp_entries([t], i[:, None]), lambda: mk.clip_grad_norm([t], 1.0)):
        with pytest.raises(TypeError):
            bad()
