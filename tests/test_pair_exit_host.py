"""A commit of the pairs' products arrives on a barrier of both CTAs, at a time of the tensor cores' own.  Each CTA
has to wait for every such arrival before it exits, or one may land in the shared memory of the next CTA on its SM.
The race cannot be provoked, so the source is read for the waits; the GPU tests of the products run them."""
import os
import re

from latency_skinny_bf16_gb300 import _build

TEXT = open(os.path.join(_build.CSRC, "linear_pair.cu")).read()
KERNEL = TEXT[TEXT.index("linear_pair_kernel(const"):TEXT.index("cudaError_t launch_as")]


def test_every_barrier_of_a_commit_is_known():
    assert set(re.findall(r"pair_commit\((\w+)", KERNEL)) == {"empty", "accf", "done"}


def test_both_producers_wait_for_the_stages_in_flight():
    producer = KERNEL[KERNEL.index("if (warp == 0) {"):KERNEL.index("} else if (warp == 1) {")]
    loop, after = producer.split("for (int k = 0; k < p.boxes; ++k)")[0], producer[producer.rindex("for (int k = 0"):]
    assert "rank" not in re.sub(r"rank \* \w+", "", loop)                 # both CTAs' producers run it
    assert "k < kStages" in after and "mbar_wait_bounded(empty(s), phase" in after and "let_land()" in after
    # the place and the phase advance as in the loop before, so that the waits are the next fills'
    step = "if (++s == kStages) {"
    assert producer.count(step) == 2 and producer.count("phase ^= 1;") == 2


def test_the_second_cta_waits_for_the_last_commit():
    end = KERNEL[KERNEL.rindex("cluster_wait_acquire();"):KERNEL.rindex("pair_dealloc(tmem)")]
    assert re.search(r"rank == 1 && \*mma_ok && !mbar_wait_bounded\(done, 0, kDrainNs\)", end)


def test_the_ring_phases_of_these_waits():
    """A barrier's parity wait passes once its phase of that parity is over; fresh barriers pass for parity 1."""
    for stages in (6, 7):
        for fills in range(0, 4 * stages):
            done = [0] * stages                     # stages given back so far
            s, phase, waited = 0, 1, [0] * stages
            for k in range(fills + stages):
                filled = len([f for f in range(min(k, fills)) if f % stages == s])
                if k >= stages or k >= fills:
                    done[s] = filled                # the wait passes only then
                assert (done[s] - 1) % 2 == phase   # what the wait asks for: the last fill's arrival
                waited[s] = filled
                s += 1
                if s == stages:
                    s, phase = 0, phase ^ 1
            assert waited == [len(range(i, fills, stages)) for i in range(stages)]
