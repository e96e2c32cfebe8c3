"""Sizes at the ends of their ranges, in the host code of a dense layer's operators."""
import os
import re
import subprocess

import pytest

from latency_skinny_bf16_gb300 import _build

CXX = os.environ.get("CXX", "g++")


def program(tmp_path, body, header="layer.h"):
    """What a C++ program with the library's headers prints."""
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(f'#include <cstdio>\n#include <initializer_list>\n#include "{header}"\nint main() {{ {body} }}\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc_path())), "include")
    subprocess.run([CXX, "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE, "-I", cuda, str(src), "-o", str(exe)],
                   check=True, timeout=300)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split()


def test_boxes_of_a_depth(tmp_path):
    """The weight's gradient sums over the tokens: as many as an int holds."""
    depths = [1, 63, 64, 65, 128, 7168, 7169, (1 << 20) + 1, 2147483584, 2147483585, 2147483600, 2147483647]
    body = "".join(f'std::printf("%d\\n", skinny::depth_boxes({d}));' for d in depths)
    assert [int(v) for v in program(tmp_path, body)] == [-(-d // 64) for d in depths]


@pytest.mark.parametrize("source", ["linear_pair.cu", "linear_tc.cu"])
def test_no_other_count_of_boxes(source):
    text = open(os.path.join(_build.CSRC, source)).read()
    assert "depth_boxes(a.depth)" in text and not re.search(r"depth\s*\+", text)


def test_single_elements_are_fetched_from_inside_their_tensor(tmp_path):
    """Views [T, H, D] from a start on and off a word's boundary, dense, with gaps, heads first."""
    body = r"""
    for (long start : {4096L, 4098L})
        for (int T = 1; T <= 3; ++T) for (int H = 1; H <= 3; ++H) for (int D = 1; D <= 5; ++D)
            for (int gap = 0; gap <= 3; ++gap) for (int order = 0; order < 2; ++order) {
                const long sh = order ? T * (D + gap) : D + gap, st = order ? D + gap : H * (D + gap);
                const unsigned long lo = start, last = start + 2 * ((T - 1) * st + (H - 1) * sh + D - 1);
                for (int t = 0; t < T; ++t) for (int h = 0; h < H; ++h) for (int d = 0; d < D; ++d) {
                    const unsigned long at = start + 2 * (t * st + h * sh + d);
                    const skinny::ElementFetch f = skinny::element_fetch(at, lo, last);
                    const bool inside = f.from >= lo && f.from + f.bytes <= last + 2, holds = f.from <= at && at + 2 <= f.from + f.bytes;
                    const bool word = f.bytes == 4 ? f.from % 4 == 0 : f.bytes == 2 && f.from == at && (at == lo || at == last);
                    const bool end = (t == 0 && h == 0) || (t == T - 1 && h == H - 1);     // where the kernel asks
                    if (!inside || !holds || !word || (f.bytes == 2 && !end)) {
                        std::printf("bad %ld %d %d %d %d %d\n", start, T, H, D, gap, order);
                        return 0;
                    }
                }
            }
    std::printf("good\n");"""
    assert program(tmp_path, body, "element_fetch.h") == ["good"]


def test_heads_fetch_their_end_elements_so():
    text = open(os.path.join(_build.CSRC, "heads.cu")).read()
    assert "kHalves && end == all ? 1 : 0" in text and "if (left <= careful || (starts && begin == 0))" in text
    assert "copy_element(dst" in text
