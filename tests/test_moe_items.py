"""The experts' kernels find the slots of a workgroup from counts that every lane of a
wave adds up in 32 bits; emulated here (CPU only) for lists that overlap, whose counts
together pass 2^32."""

import numpy as np
import pytest

MOST = 1 << 24  # kMostItems


def wrap(x):
    return (int(x) + 2 ** 31) % 2 ** 32 - 2 ** 31


def find_item(offsets, R, B, item, most):
    """(expert, its block of B slots, its blocks) of an item, None behind the last;
    32-bit counts"""
    E = len(offsets) - 1
    r0 = np.clip(offsets[:-1], 0, R).astype(np.int64)
    r1 = np.minimum(np.maximum(offsets[1:].astype(np.int64), r0), R)
    blocks = (r1 - r0 + B - 1) // B
    per = (E + 63) // 64
    mine = []
    for lane in range(64):
        n = 0
        for b in blocks[lane * per:(lane + 1) * per]:
            n = min(wrap(n + b), most)
        mine.append(n)
    upto, total = [], 0
    for n in mine:
        total = wrap(total + n)
        upto.append(total)
    if item >= total:
        return None
    owner = next(i for i in range(64) if upto[i] > item)
    rest = wrap(item - wrap(upto[owner] - mine[owner]))
    for e in range(owner * per, min((owner + 1) * per, E)):
        if rest < blocks[e]:
            return e, rest, int(blocks[e])
        rest = wrap(rest - blocks[e])
    return E, 0, 0


def overlapping(E, claim):
    """Every other expert claims `claim` slots, the same ones."""
    off = np.zeros(E + 1, np.int64)
    off[1::2] = claim
    return off


def in_range(got, E):
    e, block, blocks = got
    return 0 <= e < E and 0 <= block < blocks


E, B = 65535, 128
MOST_SLOTS = (2 ** 24 - 8) * B - 1
# a lane's 512 experts together: below 2^31 blocks, just past it, past 2^32
CLAIMS = [2 ** 20, 2 ** 29 - B, (2 ** 22 + 5) * B, 2 ** 30 + 12345, MOST_SLOTS]
ITEMS = [0, 1, 1000, 3000, 2 ** 20, 2 ** 23, 2 ** 24 - 9]


@pytest.mark.parametrize("claim", CLAIMS)
def test_overlapping_lists_give_slots_in_range(claim):
    off = overlapping(E, claim)
    for item in ITEMS:
        got = find_item(off, MOST_SLOTS, B, item, MOST)
        assert got is None or in_range(got, E)


def test_counts_without_the_stop_leave_the_range():
    """What the stop is for."""
    got = [find_item(overlapping(E, claim), MOST_SLOTS, B, item, 2 ** 40)
           for claim in CLAIMS for item in ITEMS]
    assert not all(in_range(g, E) for g in got if g is not None)


def test_every_slot_of_proper_lists_is_found_once():
    rng = np.random.default_rng(1)
    off = np.concatenate([[0], np.cumsum(rng.integers(0, 40, 200))])
    seen, item = [], 0
    while (got := find_item(off, int(off[-1]), 16, item, MOST)) is not None:
        e, block, blocks = got
        first = off[e] + 16 * block
        seen.extend(range(first, min(first + 16, off[e + 1])))
        item += 1
    assert seen == list(range(off[-1]))
