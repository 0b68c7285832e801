"""The bounded waits of windowed attention against the work that they wait for: a role without work of its own waits for as long
as the others take for what they were handed, a unit's part.  (While whole units were handed out, of up to 2^24 key tiles,
a wait could give up on one of 4 s.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_verification_gdn_gb300",
                    "csrc")
TRY_US = 3.97      # one try of a wait on a barrier that nothing arrives on, on a GB300
TILE_US = 0.82     # a key tile of one CTA, head dim 256; 0.78 at 64


def test_waits_outlast_the_longest_part():
    with open(os.path.join(CSRC, "window_tiles.cu")) as f:
        tiles = f.read()
    part_us = int(re.search(r"kPart = (\d+);", tiles)[1]) * TILE_US
    limit_us = (1 << int(re.search(r"kTries = 1u << (\d+)", tiles)[1])) * TRY_US
    assert 1000 * part_us < limit_us < 5e6
    assert re.search(r"u\.last = min\(u\.end, first \+ kPart\)", tiles)
