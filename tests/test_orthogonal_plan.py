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


def test_matrices_beyond_a_grid_go_in_several_launches(tmp_path):
    """Every matrix of a list once, in the order of the list, in launches whose blocks, elements and counts of
    matrices hold: elements of 2^31 - 1 matrices among them."""
    out = run(tmp_path, r"""
#include <cstdio>
#include <vector>
#include "newton_plan.h"
int main() {
    const int64_t full = INT32_MAX;
    int wrong = 0, launches = 0;
    for (int c : {1, 2, 4, 8})
        for (const std::vector<int64_t>& counts : std::vector<std::vector<int64_t>>{
                 {}, {0, 0}, {1}, {3, 0, 5}, std::vector<int64_t>(64, 2), std::vector<int64_t>(131, 1),
                 {full, full, full}, {1, full, full, 7}, {full / 8, 1}, {full / 8 - 1, 2, 3}}) {
            size_t at = 0;              // element and matrix that is next
            int64_t b = 0, of_launch = 0;
            int parts_of = 0;
            mk::deal(
                (int)counts.size(), 64, full / c, [&](int k) { return counts[k]; },
                [&](int part, int k, int64_t b0, int64_t n, int64_t before) {
                    while (at < counts.size() && b == counts[at]) ++at, b = 0;
                    wrong += part != parts_of || (size_t)k != at || b0 != b || n < 1 || before != of_launch;
                    b += n;
                    of_launch += n;
                    ++parts_of;
                },
                [&](int parts, int64_t n) {
                    wrong += parts != parts_of || n != of_launch || n * c > full || parts > 64;
                    of_launch = parts_of = 0;
                    ++launches;
                    return true;
                });
            while (at < counts.size() && b == counts[at]) ++at, b = 0;
            wrong += at != counts.size() || parts_of != 0;
        }
    printf("%d %d", wrong, launches > 40);
}
""")
    assert out == ["0", "1"]


def test_the_small_matrices_are_dealt_out_so():
    """The kernels for short sides take their lists by that rule."""
    with open(f"{_build.CSRC}/newton_small.cu") as f:
        text = f.read()
    assert text.count("deal(") == 1 and "INT32_MAX / c" in text and "unsigned used" not in text


def test_kernels_wait_for_what_is_in_flight_before_they_free_tensor_memory():
    """Read, not run: no wait of these kernels may run out on a GPU.  Each that frees tensor memory waits, with a
    limit, for its MMAs first, also where it has given up."""
    for name, waits in (("newton.cu", "wait_drain(done, 0"), ("newton_small.cu", "finish(bars, *abort_flag != 0")):
        with open(f"{_build.CSRC}/{name}") as f:
            kernels = f.read().split("__global__ void")[1:]
        freeing = [k for k in kernels if "tcgen05.dealloc" in k]
        assert len(freeing) == (1 if name == "newton.cu" else 2)
        for k in freeing:
            assert 0 <= k.find(waits) < k.find("tcgen05.dealloc"), name
