"""Host code of the rotation by position that no entry point shows by itself, in small programs that are
compiled here and run on the CPU."""
import os
import subprocess

from dense_tensor_decomposition_gb300 import _build


def run(tmp_path, source):
    """Standard output of a CUDA program that may include the library's sources."""
    code, program = tmp_path / "host.cu", tmp_path / "host"
    code.write_text(source)
    subprocess.run([_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-Xcicc", "-O0", "-std=c++17", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", "-o", str(program),
                    str(code)], check=True)
    return subprocess.run([str(program)], check=True, capture_output=True, text=True,
                          env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout.split()


def test_calls_of_different_sizes_leave_one_another_their_shared_memory(tmp_path):
    """What a kernel is allowed belongs to the function, not to the call: a small call between another
    thread's allowance and its launch may not take any of it back."""
    out = run(tmp_path, r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include <cuda_runtime.h>
static std::vector<int> limits;
template <typename K> static cudaError_t note(K, cudaFuncAttribute, int bytes) { limits.push_back(bytes); return cudaSuccess; }
static cudaError_t first_device(int* d) { *d = 0; return cudaSuccess; }
#define cudaFuncSetAttribute note
#define cudaGetDevice first_device
#include "rotary.cu"
int main() {
    uint64_t turns[512] = {};
    size_t most = 0;
    for (int heads : {90, 60, 95, 50}) {        // one token of some rows of 257 fp32, at an odd offset: 51 to 98 KB
        const int64_t w = 257;
        const mttkrp_rotary_tensor t{(void*)0x10004, (void*)0x1000004, heads, {0, 0, w}, {0, 0, w}};
        const mk::RotaryArgs r{1, &t, MTTKRP_F32, 1, 1, w, (void*)0x5000, 8, 0, 0, 256, turns, true, false, 1.f};
        bool taken = false;
        mk::run_dense<float, 128>(r, nullptr, taken);       // (there is no GPU for the launch)
        if (!taken) return 1;
        most = std::max(most, (size_t)(heads * w * 4 + 31) / 16 * 16);
    }
    bool kept = !limits.empty();
    for (int b : limits) kept = kept && b == limits[0] && (size_t)b >= most;
    printf("%d", kept);
}
""")
    assert out == ["1"]
