"""Turns with the one output staging buffer of the d = 128 forward kernels, without a GPU.

The two softmax slots of a CTA take turns (slot 0 of unit 0, slot 1 of unit 0, slot 0 of unit 1,
...), each turn a phase of the slot's mbarrier.  A wait on a phase's parity passes while exactly
that phase is the last one completed, so a phase that ends before a slow warp has seen the one
before leaves that warp waiting for good.  The walk of the warps is searched exhaustively here,
under the number of arrivals that each kernel's source gives the barrier.
"""
import os
import re

import pytest

from attention_forward_tiled_b200 import build as abuild

UNITS, WARPS = 5, 2  # units of a CTA, warps of a slot (two are enough for one to lag)


def arrivals(header):
    """Arrivals that end a turn, the line on which a warp passes one, and the other warps' arrival."""
    with open(os.path.join(abuild.CSRC, header)) as f:
        text = f.read()
    count = int(re.search(r"mbar_init\(BAR\(C::kBarOStage \+ i\), (\d+)\)", text).group(1))
    passed = re.findall(r"if \(([^()]*(?:\(\))?[^()]*)\) mbar_arrive\(BAR\(C::kBarOStage \+ t\)\);", text)
    return count, passed


def stuck(stored, every_warp):
    """A reachable state in which no warp can move and some has not finished, or None.

    stored[k][t]: slot t stores in unit k.  A warp's steps in a unit: 0 reads the unit (the unit
    ring lets it run at most two units ahead of the slowest), 1 waits for the turn before (a stored
    tile first needs every warp of the slot in that unit: its product waits for all their P), 2 (the
    first warp of a stored tile) waits for the others' rows.  Warps arrive for their turn when they
    pass it or, in a stored tile, have staged their rows; the first warp once the store has read
    them, at its next unit.
    """
    warps = [(t, w) for t in range(2) for w in range(WARPS)]
    need = WARPS if every_warp else 1
    start = (tuple((0, 0) for _ in warps), (0, 0), (False, False))  # places, arrivals of each slot, stores under way
    seen, todo = {start}, [start]
    while todo:
        places, count, pending = todo.pop()
        slowest = min(k for k, _ in places)
        moved = False
        for i, (t, w) in enumerate(warps):
            k, step = places[i]
            if k > UNITS or (k == UNITS and step):
                continue
            c, pend = list(count), list(pending)
            if step == 0:
                if k > slowest + 2:
                    continue
                if w == 0 and pend[t]:
                    c[t] += 1
                    pend[t] = False
                place = (k, 1) if k < UNITS else (k + 1, 0)
            elif step == 1:
                if stored[k][t] and any(places[j] < (k, 1) for j, x in enumerate(warps) if x[0] == t):
                    continue
                done = [n // need for n in c]  # turns completed
                if t == 0 and k > 0 and (done[1] & 1) == ((k - 1) & 1):
                    continue
                if t == 1 and (done[0] & 1) == (k & 1):
                    continue
                if not stored[k][t]:
                    if every_warp or w == 0:
                        c[t] += 1
                    place = (k + 1, 0)
                elif w == 0:
                    place = (k, 2)
                else:
                    if every_warp:
                        c[t] += 1
                    place = (k + 1, 0)
            else:
                if any(places[j] <= (k, 1) for j, x in enumerate(warps) if x[0] == t and x[1] != 0):
                    continue
                pend[t] = True
                place = (k + 1, 0)
            moved = True
            state = (places[:i] + (place,) + places[i + 1:], tuple(c), tuple(pend))
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(k <= UNITS for k, _ in places):
            return places
    return None


PATTERNS = {
    "second slot idle": [(True, False)] * UNITS,           # one Q tile a unit: up to 128 queries
    "nothing stored": [(False, False)] * UNITS,            # rows above the causal diagonal
    "all stored": [(True, True)] * UNITS,
    "mixed": [(False, False), (True, True), (False, False), (False, True), (True, False)],
}


def test_one_arrival_a_turn_can_strand_a_warp():
    assert stuck(PATTERNS["second slot idle"], False) and stuck(PATTERNS["nothing stored"], False)


@pytest.mark.parametrize("header", ["prefill_sm100.cuh", "window_fwd_sm100.cuh"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
def test_turns_end(header, pattern):
    count, passed = arrivals(header)
    every_warp = count == 4 and sorted(passed) == ["lane == 0", "lane == 0 && quarter != 0"]
    assert stuck(PATTERNS[pattern], every_warp) is None
