"""Prompts of linear attention where a CTA walks many chunks and several units of unlike lengths, against
the recurrence in 64 bits.  The bounds are those of test_gpu_linear_attn."""
import numpy as np
import pytest
import torch

import test_gpu_linear_attn as L
import tree_speculative_verification_gdn_gb300 as tv
from _mixer import recurrence

pytestmark = pytest.mark.gpu


def check_prompt(c, out, S, err, S0=True):
    assert not any(err)
    (o, s), (ao, as_) = recurrence(c, S0), recurrence(c, S0, absolute=True)
    n, dk = int(np.diff(c["cu"].tolist()).max()), c["q"].shape[-1]
    io = "bf16" if c["v"].dtype == torch.bfloat16 else "f32"
    L.check(out, o, ao, n, dk, io, "out")
    L.check(S, s, as_, n, dk, io, "S")


@pytest.mark.parametrize("state", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_many_chunks_repeat_themselves(dk, dv, state):
    """A chunk's scores take the place of the last chunk's, which the product with its values still reads:
    one that came early would show in the outputs, and not the same way every time."""
    c = L.make([900, 641], 8, 152, dk, dv, "bf16", state, seed=dk + dv)
    out, S, err = L.prompt(c)
    check_prompt(c, out, S, err)
    for _ in range(4):
        again, S2, _ = L.prompt(c)
        assert torch.equal(out, again) and torch.equal(S, S2)


UNLIKE = [257, 0, 1, 130, 64, 300, 128, 0, 90, 385, 5, 129]


@pytest.mark.parametrize("state", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_units_of_unlike_lengths_on_one_sm(dk, dv, state):
    # more prompts x heads than SMs: a CTA goes from one to another, over empty ones and from ragged tails
    H, T = 40, sum(UNLIKE)
    assert tv.tv_linear_attn_workspace_size(len(UNLIKE), T, 385, H, dk, dv) == 0
    c = L.make(UNLIKE, 20, H, dk, dv, "bf16", state, seed=dk - dv)
    out, S, err = L.prompt(c, max_len=385)
    check_prompt(c, out, S, err)
    again, S2, _ = L.prompt(c, max_len=385, in_place=True)
    assert torch.equal(out, again) and torch.equal(S, S2)


@pytest.mark.parametrize("state", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_segments_of_unlike_lengths_on_one_sm(dk, dv, state):
    lens, H = [3001, 129, 0, 1500, 2], 24
    assert tv.tv_linear_attn_workspace_size(len(lens), sum(lens), 3001, H, dk, dv) > 0
    c = L.make(lens, 24, H, dk, dv, "bf16", state, seed=dk + 3 * dv)
    out, S, err = L.prompt(c, max_len=3001)
    check_prompt(c, out, S, err)


@pytest.mark.parametrize("io,state", L.TYPE_SETS)
def test_prompts_that_leave_rows_out(io, state):
    # the first prompt starts behind token 0, the last one ends before T
    c = L.make([9, 150, 0, 261, 8], 2, 4, 128, 128, io, state, seed=4)
    c["cu"], c["S0"] = c["cu"][1:-1].clone(), c["S0"][1:-1].clone()
    out, S, err = L.prompt(c)
    assert not any(err)
    (o, s), (ao, as_) = recurrence(c), recurrence(c, absolute=True)
    L.check(out[9:-8], o[9:-8], ao[9:-8], 261, 128, io, "out")
    L.check(S, s, as_, 261, 128, io, "S")
    assert bool((out[:9] == 7).all()) and bool((out[-8:] == 7).all())
