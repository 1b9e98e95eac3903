"""The sampled operators' binding module on a machine with two GPUs, as far as the module
can tell: a preloaded library answers for the CUDA runtime and takes the place of the
library's entry points, which note the device that is current when they are called.  No
GPU is used and no tensor's memory is touched."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
import dense_tensor_decomposition_gb300 as mk  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <cstddef>
#include <cstdint>
static thread_local int current = 0;
static int seen = -1;
namespace c10::cuda {       // how a guard goes back to the device before it
int MaybeSetDevice(int8_t d) { current = d; return 0; }
}
extern "C" {
int cudaGetDeviceCount(int* n) { *n = 2; return 0; }
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; return 0; }
int cudaDeviceGetStreamPriorityRange(int* least, int* greatest) { *least = 0; *greatest = -1; return 0; }
int current_device() { return current; }
int device_seen() { const int d = seen; seen = -1; return d; }
int mttkrp_embedding(const void*, int64_t, int64_t, int64_t, int, const void*, int64_t, int64_t, int, float, void*,
                     int64_t, void*) { seen = current; return 0; }
size_t mttkrp_embedding_grad_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
int mttkrp_embedding_grad(const void*, int64_t, int64_t, int, const void*, int, int64_t, int64_t, int64_t, float, int,
                          void*, int, int64_t, void*, size_t, void*) { seen = current; return 0; }
int mttkrp_cp_entries(int, const int64_t*, int64_t, const void* const*, int, const void*, int64_t, int, float*,
                      void*) { seen = current; return 0; }
size_t mttkrp_cp_entries_grad_workspace_bytes(int, const int64_t*, int64_t, int64_t) { return 0; }
int mttkrp_cp_entries_grad(int, const int64_t*, int64_t, const void* const*, int, const void*, int64_t, int,
                           const float*, float* const*, void*, size_t, void*) { seen = current; return 0; }
}
"""

CALLS = r"""
import ctypes
import torch
import dense_tensor_decomposition_gb300 as mk

AT, ROOM = 0x10000, 1 << 20             # a made-up address
fake = ctypes.CDLL(None)


class Stream:
    cuda_stream = 0                     # a device's default stream


def tensor(device, *shape, dtype=torch.float32):
    where = torch.device("cuda", device)
    strides = [1] * len(shape)
    for k in range(len(shape) - 1, 0, -1):
        strides[k - 1] = strides[k] * shape[k]
    storage = torch._C._construct_storage_from_data_pointer(AT, where, ROOM)
    meta = dict(size=shape, stride=strides, dtype=dtype, storage_offset=0, device=where, nbytes=ROOM, data_ptr=AT,
                layout=torch.strided)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(meta, storage)


for device in (0, 1):
    f, x = tensor(device, 4, 8), tensor(device, 3)
    rows, idx = tensor(device, 3, 8), tensor(device, 3, dtype=torch.int32)
    at = tensor(device, 3, 2, dtype=torch.int32)
    for current in (0, 1):
        for stream in (None, Stream()):
            fake.cudaSetDevice(current)
            for call in (lambda: mk.embedding(f, idx, out=rows, stream=stream),
                         lambda: mk.embedding_grad(idx, rows, 4, out=f, stream=stream),
                         lambda: mk.cp_entries([f, f], at, out=x, stream=stream),
                         lambda: mk.cp_entries_grad([f, f], at, x, outs=[f, f], stream=stream)):
                call()
                assert fake.device_seen() == device, (device, current, stream)
                assert fake.current_device() == current
print("done")
"""


@pytest.mark.skipif(not hasattr(torch._C, "_construct_CUDA_Tensor_From_Storage_And_Metadata"),
                    reason="this PyTorch makes no tensors of a given address")
def test_calls_run_on_the_tensors_device(tmp_path):
    mk.build()
    source, fake = tmp_path / "fake.cpp", tmp_path / "libfake.so"
    source.write_text(FAKE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(fake), str(source)], check=True)
    res = subprocess.run([sys.executable, "-c", CALLS], cwd=ROOT, env={**os.environ, "LD_PRELOAD": str(fake)},
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "done" in res.stdout, res.stderr[-2000:]
