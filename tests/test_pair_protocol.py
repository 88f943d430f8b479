"""The hand-over of the pair kernel's two accumulators, as a model on CPU.

csrc/tc_pair.cu: the MMA issuer fills accumulator lt mod 2 for its unit lt = 0, 1, ... and
completes a phase of the barrier `tfull` of that accumulator; it refills one only after a phase
of `tempty`, which completes when every counted warp has arrived.  The epilogue warps and the
prefetching warp wait for tfull's phase lt / 2 by its parity alone: a test of parity cannot tell
a phase from the second one after it.  The model runs the issuer, one epilogue warp and the
prefetching warp of each CTA of a pair under random schedules; the kernel's source says whether
the prefetching warps are counted.  It checks the design, not the kernel.
"""
from __future__ import annotations

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4_gemm_error_b200", "csrc",
                      "tc_pair.cu")


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, parity):
        """mbarrier.try_wait.parity: the phase of this parity is not the one in progress."""
        return (self.phase & 1) != parity


def _run(units, seed, counted, lazy):
    """True if every role ends.  `lazy`: the prefetching warps are scheduled rarely."""
    rng = random.Random(seed)
    followers = [("epilogue", c) for c in range(2)] + [("prefetch", c) for c in range(2)]
    tfull = {r: [Barrier(1), Barrier(1)] for r in range(2)}       # one of each accumulator in either CTA
    tempty = [Barrier(2 + (2 if counted else 0)) for _ in range(2)]
    at = {"issuer": 0} | {f: 0 for f in followers}

    def ready(role):
        lt = at[role]
        if lt >= units:
            return False
        if role == "issuer":
            return tempty[lt & 1].passed((lt >> 1 & 1) ^ 1)
        return tfull[role[1]][lt & 1].passed(lt >> 1 & 1)

    while any(lt < units for lt in at.values()):
        able = [r for r in at if ready(r)]
        if not able:
            return False
        weights = [0.02 if lazy and r != "issuer" and r[0] == "prefetch" else 1.0 for r in able]
        role = rng.choices(able, weights)[0]
        lt = at[role]
        if role == "issuer":
            for r in range(2):
                tfull[r][lt & 1].arrive()
        elif role[0] == "epilogue" or counted:
            tempty[lt & 1].arrive()
        at[role] = lt + 1
    return True


def _counted():
    """Whether the source counts the prefetching warp: its constant, and an arrival after its wait."""
    text = open(SOURCE).read()
    warps = re.search(r"HAND_BACK = DEQ_WARP - EPI_WARP \+ 1;", text) and "mbar_init(tempty0 + 8 * b, 2 * HAND_BACK)" in text
    block = text[text.index("} else if (warp == 3) {"):text.index("} else if (warp >= EPI_WARP && warp < DEQ_WARP) {")]
    return bool(warps) and "mbar_arrive_remote(tempty0" in block[block.index("mbar_wait(tfull0"):]


@pytest.mark.parametrize("lazy", [False, True])
def test_every_waiter_sees_every_phase(lazy):
    for seed in range(300):
        assert _run(9, seed, _counted(), lazy), seed


def test_an_uncounted_waiter_can_be_left_behind():
    """Planted mistake: the hand-back without the prefetching warps."""
    assert not all(_run(9, seed, False, True) for seed in range(300))
