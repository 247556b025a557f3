"""No computing warp of the attention stands at a barrier that another one never reaches (a model, on the host).

The kernel's four computing warps meet at one barrier. A warp whose wait for the
next unit runs into the time limit has to leave, at any unit, while the others
got the same unit in time. A run that leaves a warp standing cannot be tried on
a GPU, so the order of waits and barriers is replayed here.
"""
import itertools
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS = 4


def warp(me, units, groups, gives_up, vote):
    """What warp `me` does: yields 's' at a plain barrier, True or False at a vote, and gets the vote's answer."""
    group = me * groups // WARPS
    for un in range(len(units) + 1):
        if un == gives_up or un == len(units):  # its wait has run out, or there are no more units
            if vote:
                yield False
            return
        kind = units[un]
        if kind == "solo" and groups > 1:
            continue  # one group's own (un % groups == group) or not this one's: no barrier either way
        if groups > 1 or kind == "shared":
            if vote:
                if not (yield True):
                    return
            elif groups > 1:
                yield "s"
        half = groups // 2
        while half >= 1:
            if half < groups // 2:
                yield "s"
            yield "s"
            half //= 2
        if kind == "shared":
            yield "s"
            yield "s"


def all_end(units, groups, gives_up, vote):
    warps = [warp(w, units, groups, gives_up.get(w), vote) for w in range(WARPS)]
    answer = [None] * WARPS
    while True:
        at = []
        for w in range(WARPS):
            try:
                at.append(warps[w].send(answer[w]))
            except StopIteration:
                at.append("left")
        if all(a == "left" for a in at):
            return True
        if any(a == "left" for a in at):
            return False  # the barrier expects four warps
        assert len({a == "s" for a in at}) == 1  # a vote never meets a plain barrier
        answer = [all(a is True for a in at) if at[0] != "s" else None] * WARPS


CASES = [list(u) for n in range(4) for u in itertools.product(("solo", "whole", "shared"), repeat=n)]


@pytest.mark.parametrize("groups", [1, 2, 4])
def test_warps_that_vote_all_leave(groups):
    for units in CASES:
        for who in itertools.chain([()], itertools.combinations(range(WARPS), 1), itertools.combinations(range(WARPS), 2)):
            for when in itertools.product(range(len(units) + 1), repeat=len(who)):
                assert all_end(units, groups, dict(zip(who, when)), vote=True), (units, who, when)


@pytest.mark.parametrize("groups", [2, 4])
def test_a_warp_that_leaves_alone_leaves_the_others_standing(groups):
    assert all_end(["whole", "solo"], groups, {}, vote=False)
    assert not all_end(["whole", "whole"], groups, {1: 1}, vote=False)


def test_the_kernel_votes_wherever_a_warp_leaves():
    with open(os.path.join(ROOT, "combine_ep_get_dispatch_gb300", "csrc", "kv_attention.cu")) as f:
        text = f.read()
    loop = text[text.index("for (int un = 0;; ++un)"):text.index("// This warp's rows.")]
    assert "mbar_wait_warp(&sh.unit_full" in loop
    leaves = [m.start() for m in re.finditer(r"\bbreak;", loop)]
    assert len(leaves) == 2 and all("all_agree(false);" in loop[max(0, at - 40):at] for at in leaves)
    # and in each unit, the first barrier of all is a vote
    rest = text[text.index("// This warp's rows."):]
    first = rest.index("all_agree(true)")
    assert "compute_sync()" not in rest[:first]
