"""Host code of the sampled operators that no entry point shows by itself, in small
programs that are compiled here and run on the CPU."""
import os
import re
import subprocess

import pytest

from dense_tensor_decomposition_gb300 import _build


def run(tmp_path, source):
    """Standard output of a CUDA program that may include the library's sources."""
    code, program = tmp_path / "host.cu", tmp_path / "host"
    code.write_text(source)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", "-o", str(program),
                    str(code)], check=True)
    return subprocess.run([str(program)], check=True, capture_output=True, text=True,
                          env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout.split()


def test_an_earlier_error_is_not_a_calls_own(tmp_path):
    """Nothing to join: success, whatever error another call left with the runtime."""
    out = run(tmp_path, r"""
#include <cstdio>
#include "sums.cuh"
int main() {
    const cudaError_t earlier = cudaSetDevice(12345);
    mk::SumArgs s{};
    s.tiles = 1;
    const cudaError_t own = mk::join<float, 4>(s, nullptr);
    printf("%d %d\n", earlier != cudaSuccess, own == cudaSuccess);
}
""")
    assert out == ["1", "1"]


@pytest.mark.parametrize("name", ["rows.cu", "sort.cu", "model.cu", "gradnorm.cu", "rows.cuh", "sums.cuh", "types.cuh"])
def test_no_loads_by_the_read_only_path(name):
    """These kernels begin before the kernel that writes what they read is done: such loads
    are not kept behind their wait for it."""
    with open(os.path.join(_build.CSRC, name)) as f:
        assert not re.search(r"__ldg|\.nc\b|__restrict__", f.read())
