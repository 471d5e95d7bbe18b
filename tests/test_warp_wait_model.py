"""Waits of whole warps. Each lane of a warp polls an mbarrier for itself; a wait
that runs out, or another role's abort, may meet lanes that have already seen the
phase complete. A model of that under random interleavings, and where the kernels
have to take one answer for the warp."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_projections_b200", "csrc")
LANES = 32


def lanes_answers(rng):
    """What each lane's wait returns, under an order of events drawn from rng:
    lanes poll in any order; the phase completes and the abort flag is raised at
    some time, in either order; a lane looks at the flag only now and then."""
    completes, aborts = rng.randrange(200), rng.randrange(200)
    answers, time = [None] * LANES, 0
    while None in answers:
        lane = rng.choice([i for i, a in enumerate(answers) if a is None])
        if time >= completes:
            answers[lane] = True
        elif rng.random() < 0.5 and time >= aborts:
            answers[lane] = False
        time += 1
    return answers


def on(answers, vote):
    """The lanes that go on to the warp-wide instruction behind the wait."""
    if vote:
        answers = [all(answers)] * LANES
    return sum(answers)


def test_lanes_own_answers_split_a_warp_and_one_vote_does_not():
    rng = random.Random(0)
    split = 0
    for _ in range(400):
        answers = lanes_answers(rng)
        split += on(answers, vote=False) not in (0, LANES)
        assert on(answers, vote=True) in (0, LANES)
        if False not in answers:  # a wait that completes for every lane stays one
            assert on(answers, vote=True) == LANES
    assert split > 20


# The barriers that whole warps wait on: the epilogues' accumulators, the ragged
# stages of the weight gradients, the ring of the 4-bit projection on both sides.
@pytest.mark.parametrize("source,barriers,count", [
    ("grouped_gemm_tc.cu", ["tfull[acc], acc_phase"], 2),
    ("grouped_gemm_bwd.cu", ["tfull[acc], acc_phase", "own[stage], par"], 2),
    ("w4_proj.cu", ["full[stage], phase", "empty[stage], phase ^ 1u"], 2),
])
def test_whole_warps_take_one_answer(source, barriers, count):
    text = re.sub(r"\s+", " ", open(os.path.join(CSRC, source)).read())
    waits = [c for c in re.findall(r"(\w+)\( ?&ctl\.([^,]+, [^,]+),", text) if c[1] in barriers]
    assert len(waits) == count
    assert all(name == "mbar_wait_warp" for name, _ in waits), waits
