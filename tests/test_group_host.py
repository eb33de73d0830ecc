"""Head groups of the masked instances (even_group and window_group in csrc/fa_internal.h), compiled here with g++
against the real header: as many heads as the measurements chose, and one where a head alone fills the L2.  No GPU is
needed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_05_gb300", "csrc")
CUDA_INC = "/usr/local/cuda/include"

EVEN = [(0, 8), (1, 8), (2, 8), (3, 8), (8, 8), (9, 8), (5, 1), (0, 1), (7, 16)]
FWD = [(4096, 1023, 128), (65536, 60000, 128), (131072, 30000, 128), (131072, 60000, 128), (131072, 130000, 128), (131072, 2 ** 31 - 1, 128),
       (262144, 200000, 64), (65536, 4095, 64), (2 ** 31 - 1, 2 ** 31 - 1, 256), (0, 0, 64)]
PROGRAM = r"""
#include "fa_internal.h"
#include <cstdio>
int main() {
    const int even[][2] = {%s}, sizes[][3] = {%s};
    for (const auto &c : even)
        std::printf("%%d\n", fa::even_group(c[0], c[1]));
    for (const auto &c : sizes)
        std::printf("%%d %%d\n", fa::window_group(c[0], c[1], 256, 4 * c[2], fa::kFwdWindowBytes, 8),
                    fa::window_group(c[0], c[1], 128, 8 * c[2], fa::kBwdWindowBytes, 4));
    return 0;
}
"""


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.isdir(CUDA_INC):
        pytest.skip("g++ or the CUDA headers are not available")
    d = tmp_path_factory.mktemp("group")
    src, exe = d / "group.cpp", d / "group"

    def table(rows):
        return ", ".join("{%s}" % ", ".join(map(str, r)) for r in rows)
    src.write_text(PROGRAM % (table(EVEN), table(FWD)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, str(src), "-o", str(exe)], check=True)
    out = list(map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()))
    n = len(EVEN)
    return dict(zip(EVEN, out[:n])), dict(zip(FWD, zip(out[n::2], out[n + 1::2])))


def test_even_groups(chosen):
    even = chosen[0]
    assert even[(0, 8)] == even[(1, 8)] == 1          # a head that fills the budget alone stays alone
    assert even[(2, 8)] == even[(3, 8)] == 2 and even[(7, 16)] == 6
    assert even[(8, 8)] == even[(9, 8)] == 8 and even[(5, 1)] == 1 and even[(0, 1)] == 1


def test_groups_under_a_window(chosen):
    both = chosen[1]
    for small in ((4096, 1023, 128), (65536, 60000, 128), (131072, 30000, 128), (65536, 4095, 64), (0, 0, 64)):
        assert both[small] == (8, 4), small
    for wide in ((131072, 60000, 128), (131072, 130000, 128), (131072, 2 ** 31 - 1, 128), (262144, 200000, 64), (2 ** 31 - 1, 2 ** 31 - 1, 256)):
        assert both[wide] == (1, 1), wide


MASKS = [((5, 0, 0), 100), ((98, 0, 4), 100), ((99, 0, 4), 100), ((99, -1, 0), 100), ((0, 0, 100), 100), ((0, 0, 99), 100), ((-1, 0, 7), 100),
         ((2 ** 31 - 1, 0, 2 ** 31 - 1), 1), ((0, 0, 0), 1), ((0, 5, 0), 2)]


def test_left_bounds_that_hide_nothing(tmp_path):
    """(left, right, sinks) and Tk: none where every key of every row is seen, and no sinks without a left bound."""
    if shutil.which("g++") is None or not os.path.isdir(CUDA_INC):
        pytest.skip("g++ or the CUDA headers are not available")
    rows = ", ".join("{%d, %d, %d, %d}" % (*m, tk) for m, tk in MASKS)
    (tmp_path / "mask.cpp").write_text(r"""
#include "fa_internal.h"
#include <cstdio>
int main() {
    const int rows[][4] = {%s};
    for (const auto &r : rows) {
        const fa::MaskSpec m = fa::effective_mask(fa::MaskSpec{r[0], r[1], nullptr, 0, r[2]}, r[3]);
        std::printf("%%d %%d %%d\n", m.left, m.right, m.sinks);
    }
    return 0;
}
""" % rows)
    exe = tmp_path / "mask"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", CUDA_INC, str(tmp_path / "mask.cpp"), "-o", str(exe)], check=True)
    out = list(map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()))
    for i, ((left, right, sinks), tk) in enumerate(MASKS):
        hides = left >= 0 and any(l < p - left and l >= sinks for p in range(min(tk, 200)) for l in range(p + 1))
        assert tuple(out[3 * i:3 * i + 3]) == ((left, right, sinks) if hides else (-1, right, 0)), (left, right, sinks, tk)
