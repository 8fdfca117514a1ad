"""Copies in flight when a cross-attention CTA gives up: which tiles a copying warp has to wait for before it ends, in a
model of its two stages, and that the sources do."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sub_byte_quantized_write_gb300", "csrc")


def run(rng, tiles, waits):
    """Issues copies into two stages until one of the other warps gives up; the copies still in flight at the end."""
    issued, landed, freed = 0, set(), set()
    gives_up = rng.randrange(0, 6 * tiles + 1)
    for tick in range(8 * tiles):
        for t in range(issued):
            if t not in landed and rng.random() < 0.4:
                landed.add(t)
        for t in sorted(landed):  # a stage is freed by what read it, after it landed, unless that has given up
            if t not in freed and tick < gives_up and rng.random() < 0.7:
                freed.add(t)
                break
        if tick >= gives_up:
            break
        if issued < tiles and (issued < 2 or issued - 2 in freed):
            issued += 1
    landed |= set(range(max(issued - waits, 0), issued))  # what is waited for
    return set(range(issued)) - landed


def test_the_last_two_tiles_are_enough_and_one_is_not():
    rng = random.Random(1)
    left = {w: sum(bool(run(rng, 9, w)) for _ in range(2000)) for w in (0, 1, 2)}
    assert left[2] == 0 and left[1] > 0 and left[0] > 0


@pytest.mark.parametrize("source,loops", [("kvq_cross16.cu", 1), ("kvq_crossq.cu", 2)])
def test_sources_wait_whoever_gave_up(source, loops):
    """The waits stand behind the copies' loop at its own depth, not inside a test of this warp's own success."""
    text = open(os.path.join(CSRC, source), encoding="utf-8").read()
    text = re.sub(r"//[^\n]*", "", text)
    found = re.findall(r"\n    for \(int u = max\(issued(?:\[\d\])? - 2, 0\); u < issued(?:\[\d\])?; \+\+u\)\s*\(void\)[^;]*FULL[^;]*;", text)
    assert len(found) == loops
