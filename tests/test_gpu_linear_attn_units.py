"""Prompts of linear attention where a CTA walks many chunks and several units of unlike lengths, against
the recurrence in 64 bits.  The bounds are those of test_gpu_linear_attn."""
import numpy as np
import pytest
import torch

import test_gpu_linear_attn as L
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
