"""A CTA that allocates tensor memory waits until its columns are free, without
a limit.  None may wait for CTAs that wait for it, so an SM holds at most two of
them, 256 of its 512 columns each: every plan asks for more than a third of an
SM's shared memory, whatever the size of its ring."""
import pytest

import latency_skinny_bf16_gb300 as sk

THIRD = 228 * 1024 // 3 - 1024      # a CTA is charged 1 KB beside what it asks for
X, W, Y = 0x7F0000000000, 0x7F1000000000, 0x7F2000000000


@pytest.mark.parametrize("stages", [0, 1, 2, 4])
@pytest.mark.parametrize("stage_k", [0, 64])
@pytest.mark.parametrize("split_k", [0, 1, 2])
def test_small_rings_keep_a_third_cta_off_the_sm(stages, stage_k, split_k):
    seen = 0
    with sk.options(backend=sk.SKINNY_BACKEND_TCGEN05, stages=stages, stage_k=stage_k, split_k=split_k):
        for M in (1, 16, 17, 33, 64):
            for N, K in ((8, 64), (64, 64), (300, 128), (2112, 512), (24576, 64), (24576, 1536)):
                try:
                    p = sk.skinny_plan_for(X, K, W, K, Y, N, M, N, K, 152)
                except sk.SkinnyError:
                    continue
                seen += 1
                assert p["backend"] == sk.SKINNY_BACKEND_TCGEN05 and p["smem_bytes"] > THIRD
    assert seen > 5
