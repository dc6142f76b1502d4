"""Arrival counts of the split-over-keys kernel, without a GPU.

The chunks of all items, end to end, are dealt to the CTAs in runs of equal length; the CTAs that
hold parts of one item count themselves in at a word, and the last clears it.  A captured launch is
replayed with the same nonce, so a count that is left behind would let the next replay join an item
before its parts are there.  The dealing is restated here; a CTA may give up in any of its parts.
"""
import os
import random
import re

import pytest

from attention_forward_tiled_b200 import build as abuild


def deal(items, run_length):
    """[(item, first chunk, end)] of each CTA's run, and every item's first chunk in the stream."""
    starts, total = [], 0
    for n in items:
        starts.append(total)
        total += n
    runs = []
    for run in range(0, total, run_length):
        end, parts = min(total, run + run_length), []
        for i, (x0, n) in enumerate(zip(starts, items)):
            if n and max(x0, run) < min(x0 + n, end):
                parts.append((i, max(x0, run) - x0, min(x0 + n, end) - x0))
        runs.append(parts)
    return runs, starts, total


class Words(dict):
    def arrive(self, word, n):
        """True for the last of n arrivals, which clears the word."""
        count = self.get(word, 0) + 1
        self[word] = 0 if count == n else count
        return count == n


def launch(items, run_length, words, gives_up=None, counts_in=True):
    """One launch, CTAs in random order; gives_up: (CTA, place of a part in its run).  Returns the items
    whose join ran before all their parts were there."""
    runs, starts, total = deal(items, run_length)
    arrived, early = {i: set() for i in range(len(items))}, []
    order = list(range(len(runs)))
    random.Random(len(items) + run_length).shuffle(order)

    for cta in order:
        gone = False
        for at, (item, a, b) in enumerate(runs[cta]):
            if gone and not counts_in:
                break
            if (a, b) != (0, items[item]):
                x0, n = starts[item], items[item]
                parts = (x0 + n - 1) // run_length - x0 // run_length + 1
                arrived[item].add(cta)
                if words.arrive(x0 // run_length, parts) and len(arrived[item]) < parts:
                    early.append(item)
            gone = gone or gives_up == (cta, at)
    return early


CASES = [([40, 3, 3, 50, 7, 0, 90], 16), ([5] * 30, 16), ([100, 1, 1, 100], 33), ([17, 15, 33, 31], 16), ([64], 16)]


@pytest.mark.parametrize("items,run_length", CASES)
def test_counts_are_cleared_whoever_gives_up(items, run_length):
    runs, _, _ = deal(items, run_length)
    for cta, parts in enumerate(runs):
        for at in range(len(parts)):
            words = Words()
            launch(items, run_length, words, (cta, at))
            assert not any(words.values())
            assert not launch(items, run_length, words)


def test_parts_left_out_would_spoil_a_replay():
    items, run_length = CASES[0]
    words = Words()
    launch(items, run_length, words, (2, 0), counts_in=False)
    assert any(words.values()) and launch(items, run_length, words)


def test_the_kernel_goes_on_to_its_last_part():
    """The loop over a run's parts ends with the run; giving up only leaves a part without chunks."""
    with open(os.path.join(abuild.CSRC, "split_sm100.cuh")) as f:
        text = f.read()
    end = text[text.index("run += cb - ca;"):text.index("do ++place.b;")]
    assert re.findall(r"if \((.*)\) break;", end) == ["run >= run_end"] and "abort" not in end
    assert re.search(r"const int mine = cb > c0 && !warp_flag\(abort_flag\) \?", text)
