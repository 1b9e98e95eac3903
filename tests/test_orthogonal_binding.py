"""The orthogonal maps' binding on a machine without a GPU: a preloaded library answers for the CUDA
runtime and takes the place of the library's entry points, which note what they are given.  No GPU is used
and no tensor's memory is touched."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(not hasattr(torch._C, "_construct_CUDA_Tensor_From_Storage_And_Metadata"),
                                reason="this PyTorch makes no tensors of a given address")

FAKE = r"""
#include <cstddef>
#include <cstdint>
#include "mttkrp.h"
static thread_local int current = 0;
static mttkrp_matrices seen[8];
namespace c10::cuda {
int MaybeSetDevice(int8_t d) { current = d; return 0; }
}
extern "C" {
int cudaGetDeviceCount(int* n) { *n = 1; return 0; }
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; return 0; }
int cudaDeviceGetStreamPriorityRange(int* least, int* greatest) { *least = 0; *greatest = -1; return 0; }
void matrices_seen(int k, int64_t* at) {
    const int64_t v[6] = {seen[k].batch, seen[k].rows, seen[k].cols, seen[k].batch_stride, seen[k].row_stride, seen[k].type};
    for (int i = 0; i < 6; ++i) at[i] = v[i];
}
size_t mttkrp_orthogonalize_workspace_bytes(int, const mttkrp_matrices*) { return 0; }
int mttkrp_orthogonalize(int n, const mttkrp_matrices* in, const mttkrp_matrices* out, int, const double*, double,
                         const float*, void*, size_t, void*) {
    for (int k = 0; k < n && k < 4; ++k) seen[k] = in[k], seen[4 + k] = out[k];
    return 0;
}
int mttkrp_rotary(int, const mttkrp_rotary_tensor*, int, int64_t, int64_t, int64_t, const void*, int, int64_t, int64_t,
                  const double*, int, int, float, int, void*) { return 0; }
}
"""

BEFORE = r"""
import ctypes
import torch
import dense_tensor_decomposition_gb300 as mk

AT, ROOM = 0x10000, 1 << 20             # a made-up address
fake = ctypes.CDLL(None)
CUDA = torch.device("cuda", 0)


def strided(shape, strides, dtype=torch.float32, at=AT):
    storage = torch._C._construct_storage_from_data_pointer(at, CUDA, ROOM)
    meta = dict(size=tuple(shape), stride=tuple(strides), dtype=dtype, storage_offset=0, device=CUDA, nbytes=ROOM, data_ptr=at,
                layout=torch.strided)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(meta, storage)


def tensor(*shape, **more):
    strides = [1] * len(shape)
    for k in range(len(shape) - 1, 0, -1):
        strides[k - 1] = strides[k] * max(shape[k], 1)
    return strided(shape, strides, **more)


def matrices(k):
    v = (ctypes.c_int64 * 6)()
    fake.matrices_seen(k, v)
    return list(v)


def raises(kind, call):
    try:
        call()
    except kind:
        return True
    return False

"""


def run(tmp_path, calls):
    mk.build()
    source, fake = tmp_path / "fake.cpp", tmp_path / "libfake.so"
    source.write_text(FAKE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{os.path.join(ROOT, 'include')}", "-o", str(fake),
                    str(source)], check=True)
    res = subprocess.run([sys.executable, "-c", BEFORE + calls + "\nprint('done')\n"], cwd=ROOT,
                         env={**os.environ, "LD_PRELOAD": str(fake)}, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "done" in res.stdout, res.stderr[-2000:]


def test_no_matrices_in_any_dimension(tmp_path):
    """A dimension of size 0 anywhere in front leaves nothing to do, whatever the strides; others are as before."""
    run(tmp_path, r"""
for shape in ((0, 5, 5), (2, 0, 5, 5), (0, 2, 5, 5), (3, 0, 2, 5, 5), (2, 3, 0, 5), (2, 3, 5, 0)):
    x, y = tensor(*shape), tensor(*shape, at=AT + ROOM)
    assert mk.orthogonalize(x, outs=y) is y, shape
    batch, rows, cols = matrices(0)[:3]
    assert batch * rows * cols == 0 and (rows, cols) == shape[-2:]
x, y = tensor(2, 3, 5, 4), tensor(2, 3, 5, 4, at=AT + ROOM)
mk.orthogonalize(x, outs=y)
assert matrices(0) == [6, 5, 4, 20, 4, 0] and matrices(4) == matrices(0)
apart = strided((2, 3, 5, 4), (100, 20, 4, 1))
assert raises(ValueError, lambda: mk.orthogonalize(apart, outs=y))
""")


def test_results_are_allocated_through_the_dispatcher(tmp_path):
    """As every other operator's, so that a dispatch mode (and the filling of new memory in deterministic
    mode) sees them: results of the tensors' layout, dense or not."""
    run(tmp_path, r"""
from torch.utils._python_dispatch import TorchDispatchMode


class Allocations(TorchDispatchMode):
    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        name = func._schema.name
        if name in ("aten::empty", "aten::empty_strided"):
            made.append(strided(args[0], args[1]) if name == "aten::empty_strided" else tensor(*args[0]))
            return made[-1]
        return func(*args, **(kwargs or {}))


freqs, at = mk.rotary_frequencies(16), tensor(5, dtype=torch.int64)
made = []
for x in (tensor(5, 16), tensor(5, 3, 16), strided((5, 3, 16), (16, 80, 1)), strided((5, 3, 16), (60, 20, 1)),
          strided((5, 3, 16), (48, 0, 1))):
    made.clear()
    with Allocations():
        y = mk.rotary(x, at, freqs)
    assert len(made) == 1 and y is made[0], x.stride()
    dense = x.stride() not in ((60, 20, 1), (48, 0, 1))
    assert y.stride() == (x.stride() if dense else (48, 16, 1))
""")


def test_all_tensors_of_a_matrix_lie_alike(tmp_path):
    """Rows consecutive in all of them or columns in all of them; else the call is refused, before the library
    is called."""
    run(tmp_path, r"""
rows = lambda k: strided((6, 4), (4, 1), at=AT + k * ROOM)
columns = lambda k: strided((6, 4), (1, 6), at=AT + k * ROOM)
for kinds in range(1, 15):
    made = [columns(k) if kinds >> k & 1 else rows(k) for k in range(4)]
    assert raises(ValueError, lambda: mk.orthogonal_step(made[0], made[1], made[2], 0.1, outs=made[3])), kinds
    if kinds in (1, 2):
        assert raises(ValueError, lambda: mk.orthogonalize(made[0], outs=made[1])), kinds
x, y = columns(0), columns(1)
assert mk.orthogonalize(x, outs=y) is y and matrices(0) == [1, 4, 6, 24, 6, 0]
""")
