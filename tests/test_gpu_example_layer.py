"""The linear-attention layer of ``examples/`` end to end: prompts, then tokens from a captured graph.

Both ways round the same bf16 values at the same places: projection, mixer output, gated norm, block
output and next norm, each at most half a step (2^-8) off the exact value, five of them, each carried
on by factors of order one; two ways, so at most 10 * 2^-8 of a value, and values of up to 4.5 times
their root mean square occur among some 20000 normal ones: 0.18.  The fp32 states of two ways differ by
the bf16 inputs' products only through the matrix units' operands (2^-14) and the projections' sums,
whose last bits may differ with the number of rows: one bf16 step (2^-7) of a key or value, about
2^-7 / sqrt(3) of the state if every one of them differed.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("linear_attention_layer",
                                                  os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kw", [{}, dict(lengths=(5, 260), tokens=3, heads=4, key_heads=4, dk=64, dv=64, width=256)])
def test_tokens_continue_prompts(kw):
    outputs, states = _example().serve(**kw)
    assert outputs <= 10 * 2.0 ** -8 * 4.5
    assert states <= 2.0 ** -7 / 3 ** 0.5
