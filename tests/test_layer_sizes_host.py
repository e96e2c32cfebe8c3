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
    src.write_text(f'#include <cstdio>\n#include "{header}"\nint main() {{ {body} }}\n')
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
