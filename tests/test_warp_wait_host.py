"""Host-side model of a role's warp in the tensor-core kernels of moe_linear when a wait runs out in one lane only.

The lanes poll an mbarrier one by one.  A lane may reach its limit just before the phase completes, while the others see it
complete.  What follows a wait (elect.sync, tcgen05.ld, __syncwarp) needs every lane of the warp: if a lane leaves its loop
alone, it waits at the __syncwarp behind the role for lanes that wait for it at elect.sync, with no limit.  A vote over
the wait's result makes the lanes leave together."""
import random
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).parent.parent / "moe_expert_ffn_rms_gb300" / "csrc"


def run(stages, lanes, seed, vote):
    """"done" or "stuck" for one warp, each lane a coroutine that yields what it waits for."""
    rng = random.Random(seed)
    lands = [rng.randint(0, 12) for _ in range(stages)]  # polls until a stage's phase completes
    clock = [0]
    abort = [False]

    def wait(k, limit):
        """One lane's mbar_wait: True, or False after its limit or another's."""
        n = 0
        while clock[0] < sum(lands[:k + 1]):
            if abort[0] or n >= limit:
                abort[0] = True
                return
            n += 1
            yield "poll"
        return

    def lane():
        for k in range(stages):
            yield from wait(k, rng.choice((3, 8, 100)))
            passed = clock[0] >= sum(lands[:k + 1])
            if vote:
                passed = yield ("vote", passed)
            if not passed:
                break
            yield "elect"
        yield "syncwarp"

    warp = {i: lane() for i in range(lanes)}
    at = {i: next(g) for i, g in warp.items()}
    for _ in range(10000):
        if not at:
            return "done"
        polling = [i for i, w in at.items() if w == "poll"]
        if polling:  # in any order, and phases complete in between
            i = rng.choice(polling)
            clock[0] += rng.random() < 0.5
            at[i] = next(warp[i])
            continue
        kinds = {w if isinstance(w, str) else w[0] for w in at.values()}
        if len(kinds) > 1:
            return "stuck"  # lanes at different collective instructions, each waiting for the others
        result = all(w[1] for w in at.values()) if kinds == {"vote"} else None
        after = {}
        for i in at:
            try:
                after[i] = warp[i].send(result)
            except StopIteration:
                pass
        at = after
    return "stuck"


@pytest.mark.parametrize("stages,lanes", [(1, 2), (4, 4), (9, 8)])
def test_lanes_that_vote_leave_together(stages, lanes):
    assert all(run(stages, lanes, seed, vote=True) == "done" for seed in range(400))


def test_lanes_that_leave_alone_get_stuck():
    assert any(run(4, 4, seed, vote=False) == "stuck" for seed in range(400))


def test_every_wait_of_a_warp_in_the_products_is_voted_on():
    src = (CSRC / "linear.cu").read_text()
    waits = re.findall(r".*\b(?:mbar_wait|producer_tail|accumulator_tail)\(.*", src)
    assert len(waits) == 5 and all("__all_sync(0xffffffffu, " in w for w in waits), waits
    assert len(re.findall(r"\bok = warp_wait\(", src)) == 9
