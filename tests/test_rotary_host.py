"""Host code of the rotation by position that no entry point shows by itself, in small programs that are
compiled here and run on the CPU."""
import ctypes
import os
import subprocess

import pytest

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


def test_frequencies_become_turns_to_the_last_bit(tmp_path):
    """Radians of every size and sign in units of 2^-64 turn, against whole numbers: pi to 1200 bits by Machin's
    formula.  Half a unit off at most, so that positions of 2^40 turn by what the frequency says within 2^-25."""
    def arctan_of_inverse(n, one):
        term = total = one // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total

    bits = 1200
    one = 1 << bits
    two_pi = 8 * (4 * arctan_of_inverse(5, one) - arctan_of_inverse(239, one))
    values = [0.0, 1.0, -1.0, 0.5, -0.37, 1e-5, 2 * 3.141592653589793, 7.5, 1e-12, 1e-19, -1e-19, 3e-20, 1e-300, 5e-324, 1e10,
              -1e10, 12345678.9, 2.0 ** 52 + 1, 1e18, -(2.0 ** 63), 1.8e19, 2.0 ** 64 * (1 - 2.0 ** -53)]
    values += [10000.0 ** (-i / 64) for i in range(64)] + [-(500000.0 ** (-i / 64)) for i in range(64)]
    code, program = tmp_path / "turns.cpp", tmp_path / "turns"
    code.write_text(r"""
#include <cinttypes>
#include <cstdio>
#include "turns.h"
int main() {
    const double all[] = {""" + ", ".join(v.hex() for v in values) + r"""};
    for (double f : all) printf("%" PRIu64 " ", mk::turns_of(f));
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{_build.CSRC}", "-o", str(program), str(code)], check=True)
    got = [int(x) for x in subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split()]
    assert len(got) == len(values)
    for f, turns in zip(values, got):
        numerator, denominator = f.as_integer_ratio()
        want = numerator * one * one * 2 ** 64 // (denominator * two_pi)        # turns 2^64, times `one`
        off = (turns * one - want) % (one << 64)
        off = min(off, (one << 64) - off)
        assert off * 2 <= one + (one >> 30), (f, turns)


def test_frequencies_out_of_range_are_refused():
    """2^64 radians a position and more, which 53 bits say nothing about (nothing is dereferenced)."""
    mk = pytest.importorskip("dense_tensor_decomposition_gb300")
    mk.build()
    lib = mk.load_library()
    tensors = (ctypes.c_int64 * 9)()            # no heads: nothing to do once the frequencies are taken
    for f, code in ((2.0 ** 64, 1), (-(2.0 ** 70), 1), (1e308, 1), (2.0 ** 64 * (1 - 2.0 ** -53), 0), (-1e19, 0)):
        freqs = (ctypes.c_double * 1)(f)
        assert lib.mttkrp_rotary(1, tensors, 0, 1, 1, 2, 0x1000, 8, 0, 0, freqs, 2, 0, 1.0, 0, None) == code, f


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_frequencies_by_parts_need_waves_that_get_longer(base):
    mk = pytest.importorskip("dense_tensor_decomposition_gb300")
    pytest.importorskip("torch")
    with pytest.raises(ValueError):
        mk.rotary_frequencies(8, base, "parts", 4.0, 1000)
    assert len(mk.rotary_frequencies(8, base, "turns", 4.0, 1000)) == len(mk.rotary_frequencies(8, base)) == 4
