"""The exchange between the two key streams of the many-row attention kernel, on the CPU: every order in which the streams'
steps can happen is walked, with the barriers as the kernel has them, and no read may find another item's value."""
import itertools
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_gated_delta_02_gb300", "csrc",
                      "cache4_attn_tc.cu")

# A stream's steps per item, in order: WAIT for its last product, WRITE its maximum and sum, wait for the PAIR, READ the
# other's, FREE the accumulators.
WAIT, WRITE, PAIR, READ, FREE = range(5)


def stale_reads(tiles, places):
    """(item, item found) of every read that can find another item's value.  tiles[i]: the streams with a key tile in item i."""
    n, seen, bad = len(tiles), set(), set()
    todo = [((0, 0), (None,) * (2 * places))]  # steps done by each stream, and the item whose values each place holds
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        done, held = state
        for t in (0, 1):
            item, step = divmod(done[t], 5)
            if item == n:
                continue
            at, other = item % places * 2 + t, item % places * 2 + 1 - t
            new = held
            # products of an item's first tiles wait until both streams have read the last item's accumulators;
            # a stream without a tile finds the phase that it waits for long over
            if step == WAIT and t in tiles[item] and item and min(done) < (item - 1) * 5 + FREE + 1:
                continue
            if step == WRITE:
                new = held[:at] + (item,) + held[at + 1:]
            if step == PAIR and min(done) <= item * 5 + WRITE:  # (each has arrived once it has written)
                continue
            if step == READ and held[other] != item:
                bad.add((item, held[other]))
            todo.append((tuple(d + (s == t) for s, d in enumerate(done)), new))
    return bad


def places():
    with open(SOURCE) as f:
        found = re.search(r"PAIR_PLACES = (\d+);", f.read())
    return int(found.group(1)) if found else 1


@pytest.mark.parametrize("items", [4])
def test_no_stream_reads_another_items_maximum_and_sum(items):
    """One-tile items of either stream and items of several tiles, in every order."""
    for tiles in itertools.product(((0,), (1,), (0, 1)), repeat=items):
        assert not stale_reads(tiles, places()), tiles


def test_the_model_finds_the_fault_of_a_single_place():
    assert stale_reads(((0, 1), (0,)), 1) == {(0, 1)}
    assert not stale_reads(((0, 1),) * 4, 1)  # with tiles for both the next item's products order them
