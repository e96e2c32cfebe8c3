"""A dense layer's kernels run beside the kernel before them, so no load of theirs may take its memory for constant:
the non-coherent path is only for what nothing writes during the whole kernel."""
import os
import re

import pytest

from latency_skinny_bf16_gb300 import _build


@pytest.mark.parametrize("source", ["heads.cu", "linear_tc.cu", "linear_pair.cu", "linear_dz.cu", "linear_empty.cu",
                                    "rows_pack.cu", "product.cuh", "act.cuh"])
def test_no_load_by_the_constant_path(source):
    text = open(os.path.join(_build.CSRC, source)).read()
    assert not re.search(r"__ldg\(|\.nc\b|ldg_stream|__restrict__", text)
