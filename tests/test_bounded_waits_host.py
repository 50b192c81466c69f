"""The coded product's bounded waits (not gpu): a wait that gives up must not leave
other warps of its block behind at a named barrier.

The result warps' steps are read from the kernel's source and played through for every
combination of what their waits can return: a wait that gives up in one warp may have
passed in another, whose phase ended in the meantime."""
import itertools
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exl3_trellis_weight_gb300", "csrc")

WARPS = 4
STEPS = {
    "wait": r"\bbar_wait\(acc_full",              # a warp's own wait for the accumulator
    "vote": r"\bbar_all\(1 \+ og, 128",           # the group's barrier, joining the warps' outcomes
    "meet": r"\bbar\.sync %0, 128;",              # the group's barrier
    "leave": r"if \(!ok\)\s*break;",
}


def result_steps():
    """Order of the steps in one turn of the result warps' loop over accumulators."""
    with open(os.path.join(CSRC, "linear_product.cu")) as f:
        text = f.read()
    role = text[text.index("// ---- results ----"):text.index("// ---- activations ----")]
    found = [(m.start(), name) for name, pat in STEPS.items() for m in re.finditer(pat, role)]
    return [name for _, name in sorted(found)]


def all_end(steps, outcomes):
    """Whether all warps come to the end when warp w's wait returns outcomes[w]."""
    at, ok, done = [0] * WARPS, [True] * WARPS, [False] * WARPS
    while True:
        moved = False
        for w in range(WARPS):
            while not done[w] and at[w] < len(steps) and steps[at[w]] in ("wait", "leave"):
                if steps[at[w]] == "wait":
                    ok[w] = outcomes[w]
                elif not ok[w]:
                    done[w] = True
                at[w] += 1
                moved = True
            if at[w] == len(steps):
                done[w] = True
        if all(done):
            return True
        here = {None if done[w] else steps[at[w]] for w in range(WARPS)}
        if None not in here:                      # the barrier counts 128 threads, whoever they are
            if here == {"vote"}:
                ok = [all(ok)] * WARPS
            at = [a + 1 for a in at]
            moved = True
        if not moved:
            return False


def test_result_warps_leave_together():
    steps = result_steps()
    assert "wait" in steps and "meet" in steps and "leave" in steps
    for outcomes in itertools.product((True, False), repeat=WARPS):
        assert all_end(steps, outcomes), (steps, outcomes)


def test_the_replay_finds_warps_left_behind():
    assert all_end(["meet"], [True] * WARPS)
    assert not all_end(["wait", "leave", "meet"], [True, True, True, False])
    assert all_end(["wait", "vote", "leave", "meet"], [True, True, True, False])
