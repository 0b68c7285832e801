"""The sampled rounds of ``examples/`` end to end: prompts, drafted tokens one at a time, chains, acceptance, the caches
written again after a refusal.

Both ways round the same bf16 values at the same places: queries, keys, values, weights and outputs, five of them, each at
most half a step (2^-8) off, uniform within it, two ways: sqrt(5 * 2 / 3) 2^-8 of the norm if independent.  Queries and
keys come from sums whose last bits may differ with the number of rows, and a score of up to 3 carries their 2^-8 into its
weight: 3 sqrt(2) 2^-8.  Together 4.6 * 2^-8; twice that is allowed."""
import importlib.util
import os

import pytest

from oracle import window as O

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("sampled_round", os.path.join(ROOT, "examples", "sampled_round.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kw", [{}, dict(lengths=(300, 17, 5, 64), hd=128, Hq=8, Hkv=2, window=0, sinks=0, drafts=7, rounds=4),
                                dict(lengths=(90, 200), hd=256, Hq=16, Hkv=1, window=33, sinks=20, drafts=2, rounds=5, seed=9)])
def test_rounds_commit_what_whole_prompts_would_see(kw):
    lengths = []

    def watch(parents, tokens, p, q, u, path, length, after):
        for b in range(len(length)):
            want = O.accept_sample(parents[b].tolist(), tokens[b].tolist(), p[b].double().cpu().numpy(),
                                   q[b].double().cpu().numpy(), u[b].cpu().numpy(), path.shape[1])
            n = int(length[b])
            assert (path[b, :n].tolist(), int(after[b])) == want and (path[b, n:] == -1).all()
            lengths.append(n)

    said, off = _example().serve(watch=watch, **kw)
    assert off <= 2 * 4.6 * 2.0 ** -8
    assert min(lengths) < max(lengths)      # some drafted tokens stood and some did not
    n = kw.get("lengths", (40, 1, 133))
    assert sum(len(s) for s in said) == sum(n) + sum(lengths)
