"""Host-side model of the row stages of the streaming norm kernels (csrc/norm.cu: layernorm_stream_kernel and
norm_grad_stream_kernel) when waits run out.

Thread 0 sends row n of its CTA to stage n % S; every thread waits for each row by itself, with a limit, reads the
stage, and after a barrier thread 0 sends for row n + S if its own waits have passed so far.  A wait may run out in one
thread just before the copy lands and pass in the others.  What has to hold whatever the order:
  - the status word says so if any thread's wait ran out: so every thread reports its own,
  - no copy is in flight when the CTA ends (the next CTA owns the shared memory then): so thread 0 waits at the end for
    the last copy into each stage if a wait of its own ran out,
  - no stage is sent for or written while a copy is on its way to it or a thread has still to read it."""
import random
import re
from pathlib import Path

import pytest


def run(rows, S, threads, seed, every_thread_reports=True, drain=True):
    """The faults of one CTA's life, as a set of names."""
    rng = random.Random(seed)
    faults, flight, landed = set(), {}, set()  # flight: row -> time left
    last, abort, any_failed = -1, False, False
    ok = [True] * threads

    def tick():
        for n in list(flight):
            flight[n] -= 1
            if flight[n] <= 0:
                del flight[n]
                landed.add(n)

    def send(n):
        nonlocal last
        if any(m % S == n % S for m in flight):
            faults.add("a stage sent for while its copy was in flight")
        flight[n] = rng.choice((1, 2, 3, 12, 40))
        last = n

    for n in range(min(S, rows)):
        send(n)
    for n in range(rows):
        order = list(range(threads))
        rng.shuffle(order)
        for t in order:
            left = rng.choice((2, 4, 8, 64))  # the limit that this thread's wait still has
            while n not in landed:
                if abort or left == 0:
                    abort, any_failed = True, True
                    ok[t] = False
                    break
                left -= 1
                tick()
            if rng.random() < 0.3:
                tick()  # the copy may land between one thread's last look and the next one's
            if n in landed and any(m % S == n % S for m in flight):
                faults.add("a stage written while a thread reads it")
        if ok[0] and n + S < rows:  # behind the barrier of the row's sums
            send(n + S)
    flagged = not all(ok) if every_thread_reports else not ok[0]
    if drain and not ok[0]:
        for n in range(max(0, last + 1 - S), last + 1):
            while n in flight:
                tick()
    if any_failed and not flagged:
        faults.add("a wait that ran out is not reported")
    if flight:
        faults.add("a copy in flight at the end")
    return faults


CASES = [(1, 1, 2), (5, 2, 3), (9, 3, 4), (20, 8, 4), (4, 8, 3)]


@pytest.mark.parametrize("rows,S,threads", CASES)
def test_waits_that_run_out_are_reported_and_copies_waited_for(rows, S, threads):
    for seed in range(500):
        assert not run(rows, S, threads, seed)


def test_thread_0_alone_is_not_enough():
    seen = set().union(*(run(*c, seed, every_thread_reports=False, drain=False) for c in CASES for seed in range(500)))
    assert seen == {"a wait that ran out is not reported", "a copy in flight at the end"}


def test_the_kernels_end_as_the_model_does():
    src = (Path(__file__).parent.parent / "moe_expert_ffn_rms_gb300" / "csrc" / "norm.cu").read_text()
    kernels = [b for b in re.split(r"(?m)^template <|^}", src) if "mbar_init(&full[s]" in b]
    assert len(kernels) == 2
    for b in kernels:
        assert "s_last = t;" in b and "stream_end(ok, full, S, s_last, status);" in b
        assert "flag_status" not in b  # no thread's own rule beside it
