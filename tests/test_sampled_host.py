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


def test_the_sort_fits_the_sms_there_are(tmp_path):
    """Its CTAs wait for one another: no more of them than SMs, together with all tokens, in no
    larger a workspace than the one asked for."""
    out = run(tmp_path, r"""
#include <cstdio>
#include "sort.cu"
int main() {
    for (int sms : {8, 20, 66, 132, 148, 152})
        for (int d : {1, 2, 3, 6, 8})
            for (int64_t n : {1, 1023, 20000, 70001, 262144, 622593, 1300003, 40000000})
                for (int64_t rows : {1, 900, 1 << 20}) {
                    mk::IndexArgs x{nullptr, 4, d, n, d, {}};
                    for (int m = 0; m < d; ++m) x.rows[m] = rows;
                    const mk::SortPlan p = mk::plan_sort(x, 16, sms), most = mk::plan_sort(x, 16, mk::kSms);
                    if (p.ctas < 1 || p.ctas * d > sms || p.ctas * p.per_cta < n || p.total() > most.total())
                        printf("%d_%d_%lld ", sms, d, (long long)n);
                }
    printf("done");
}
""")
    assert out == ["done"]
