"""The bounded waits of windowed attention against the longest unit that the call accepts: a role without work of its own
waits for as long as the others take for a unit."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_verification_gdn_gb300",
                    "csrc")
TRY_US = 3.97      # one try of a wait on a barrier that nothing arrives on, on a GB300
TILE_US = 0.82     # a key tile of one CTA, head dim 256; 0.78 at 64


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_waits_for_a_unit_outlast_the_longest_one():
    tiles = text("window_tiles.cu")
    most = 1 << int(re.search(r"max_blocks > \(1 << (\d+)\)\) return TV_ERR_UNSUPPORTED", text("tv_api.cu"))[1])
    keys = int(re.search(r"static constexpr int KT = (\d+);", tiles)[1])
    unit_us = most * 16 // keys * TILE_US
    inside, units = (1 << int(re.search(name + r" = 1u << (\d+)", tiles)[1]) for name in ("kTries", "kUnitTries"))
    assert unit_us < 0.5 * units * TRY_US < 20e6        # twice as long, and not much more
    assert inside * TRY_US < 5e6
    for barrier in ("unit_full", "unit_empty"):
        waits = re.findall(r"wait_for\(&bar\." + barrier + r"\[[^;]*;", tiles)
        assert waits and all("kUnitTries" in w for w in waits)
