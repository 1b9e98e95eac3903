"""How the orthogonalisation deals its work out: the rules of the library's host code, walked over
sizes in small programs that are compiled here and run on the CPU."""
import subprocess

from dense_tensor_decomposition_gb300 import _build


def run(tmp_path, source):
    """Standard output of a C++ program that includes the library's headers."""
    code, program = tmp_path / "host.cpp", tmp_path / "host"
    code.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", "-o", str(program), str(code)],
                   check=True)
    return subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout.split()


def test_every_share_of_an_item_has_a_step(tmp_path):
    """S that a cluster's CTAs share: no matrix of the list has fewer steps than there are shares, however
    long another one is, and the shares are all of its steps."""
    out = run(tmp_path, r"""
#include <cstdio>
#include "newton_plan.h"
struct List {
    int n, split;
    uint32_t items;
    mk::Shape shape[mk::kTable];
};
int main() {
    long empty = 0, split = 0;
    auto walk = [&](int sms, bool full, std::initializer_list<mk::Shape> shapes) {
        List p{};
        for (const mk::Shape& s : shapes) p.shape[p.n++] = s;
        mk::number_items(p, mk::kGram, 1, full, sms);
        split += p.split > 1;
        for (int k = 0; k < p.n; ++k) {
            const int steps = mk::Grid(p.shape[k]).steps(mk::kGram);
            int sum = 0;
            for (int share = 0; share < p.split; ++share) {
                const int here = mk::share_begin(steps, share + 1, p.split) - mk::share_begin(steps, share, p.split);
                empty += here < 1;
                sum += here;
            }
            empty += sum != steps;
        }
    };
    auto one = [](int rows, int cols, int count = 1) { return mk::Shape{0, rows, cols, count, {0, 0}}; };
    for (int sms : {132, 148, 152})
        for (bool full : {false, true}) {
            walk(sms, full, {one(512, 2000), one(160, 160)});
            walk(sms, full, {one(2000, 150), one(150, 150, 2)});
            walk(sms, full, {one(2500, 160), one(160, 160)});
            walk(sms, full, {one(768, 1024), one(192, 192)});
            for (int n = 129; n <= 3000; n += 2) {
                walk(sms, full, {one(n, n)});
                for (int m : {129, 160, 192, 193, 256, 257, 320, 500}) {
                    walk(sms, full, {one(m, n)});
                    walk(sms, full, {one(n, m), one(m, m)});
                    walk(sms, full, {one(m, m, 3), one(m, n), one(192, 129)});
                }
            }
        }
    printf("%ld %d", empty, split > 1000);
}
""")
    assert out == ["0", "1"]
