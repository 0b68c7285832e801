"""How exactly an fp32 state comes out of bf16 prompts, as a fraction of its norm.

The bound, for C chunks of 128 tokens and u = 2^-24:
  * a chunk's own sum takes 24 accumulations in the matrix units (three parts of the decayed keys, 16
    tokens at a time).  Each cuts towards zero, by half a unit of the last place on average, which is
    0.36 * 2^-23 of a value: 24 * 0.36 * 2^-23, were every partial sum as large as the whole;
  * a token's decay to the chunk's end is a hardware power of two, good to 2^-22;
  * what a state leaves out when it is rounded, by its parts between chunks and once at the end: sqrt(C) u.
    (A state rounded to a float by every chunk does not keep to that: 94 decays of 1 - 2^-17 each round an
    element the same way, and came to 2.2e-6.)
  * a decay e^-x is off by the last places of the logarithm, its product and its sum, 2^-22 x, or by 2^-22
    for a chunk that decays below a half, where x >= 0.69: 1.45 * 2^-22 x.  Tokens that keep coming are
    about x = 1 old in the norm; a state that is all old is as old as the prompt (looked at up to e^-20).
A cut prompt's segments are sums of their chunks' sums, added in fp32: the third again, not more often.
A state to which nothing is added has the last two only.  No part of it depends on how large the state is
beside what is added, or on which tokens add anything.
"""
import pytest
import torch

import test_gpu_linear_attn as L
import tree_speculative_verification_gdn_gb300 as tv
from _mixer import recurrence

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
KINDS = ["normal", "positive", "no keys", "no values", "first token", "every other block", "large start"]
ALL_OLD = ["no keys", "no values", "first token", "large start"]
ONE = torch.tensor(1.0)
DECAYS = [1.0, float(torch.nextafter(ONE, torch.tensor(0.0))), 1 - 1e-6, 1 - 1e-5, 0.9999, 0.999, 0.9]


def bound(chunks, age=1.0, adds=True):
    return (24 * 0.36 * 2.0 ** -23 + 2.0 ** -22 if adds else 0.0) + chunks ** 0.5 * U + 1.45 * 2.0 ** -22 * age


def make(T, H, dk, dv, kind, io=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(T + dk)
    q, k, v = (torch.randn(T, n, d, generator=g, device=DEV) for n, d in ((1, dk), (1, dk), (H, dv)))
    S0 = 0.1 * torch.randn(1, H, dv, dk, generator=g, device=DEV)
    if kind == "positive":
        k, v = k.abs(), v.abs()
    k = torch.nn.functional.normalize(k, dim=-1)
    if kind == "no keys":
        k.zero_()
    if kind == "no values":
        v.zero_()
    if kind == "first token":
        k[1:] = 0
    if kind == "every other block":
        k[torch.arange(T, device=DEV) // 64 % 2 == 1] = 0
    if kind == "large start":
        S0 *= 1e8
    alpha = torch.tensor(DECAYS, device=DEV)[torch.arange(H, device=DEV) % len(DECAYS)]
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    return dict(q=q.to(io), k=k.to(io), v=v.to(io), alpha=alpha, cu=cu, S0=S0)


def check(c, S, kind, heads):
    T = c["k"].shape[0]
    k, far = c["k"][:, 0].double(), torch.arange(T - 1, -1, -1, dtype=torch.float64, device=DEV)
    for h in heads:
        a = c["alpha"][h].double()
        want = (c["v"][:, h].double() * (a ** far)[:, None]).T @ k + c["S0"][0, h].double() * a ** T
        age = min(20.0, float(-T * a.log())) if kind in ALL_OLD else 1.0
        off = float((S[0, h].double() - want).norm() / want.norm().clamp_min(1e-30))
        assert off <= bound(-(-T // 128), age, kind not in ("no keys", "no values")), (h, float(a), off)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64)])
def test_state_of_a_long_prompt_in_one_piece(kind, dk, dv):
    T, H = 12000, 152
    assert tv.tv_linear_attn_workspace_size(1, T, T, H, dk, dv) == 0
    c = make(T, H, dk, dv, kind)
    _, S, err = L.prompt(c)
    assert not any(err)
    check(c, S, kind, list(range(7)) + [150])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,dk,dv", [(12000, 128, 128), (32768, 128, 128), (9001, 64, 128), (9001, 128, 64), (9001, 64, 64)])
def test_state_of_a_long_prompt_in_segments(kind, T, dk, dv):
    H = 7
    assert tv.tv_linear_attn_workspace_size(1, T, T, H, dk, dv) > 0
    c = make(T, H, dk, dv, kind)
    _, S, err = L.prompt(c)
    assert not any(err)
    check(c, S, kind, range(H))


def test_states_of_ragged_prompts_in_segments():
    lens = [3001, 6, 7, 849, 0, 666, 10, 3]
    c = L.make(lens, 4, 8, 128, 128, "bf16", "f32", seed=4)
    assert tv.tv_linear_attn_workspace_size(8, sum(lens), 3001, 8, 128, 128) > 0
    out, S, err = L.prompt(c, max_len=3001)
    want = torch.from_numpy(recurrence(c)[1]).to(DEV)
    assert not any(err)
    for b, n in enumerate(lens):
        assert float((S[b].double() - want[b]).norm() / want[b].norm()) <= bound(-(-n // 128), adds=n > 0), b
    again, S2, _ = L.prompt(c, max_len=3001)
    assert torch.equal(out, again) and torch.equal(S, S2)


def test_states_of_many_prompts_with_decays_per_token():
    c = L.make([600] * 10 + [128, 300], 8, 16, 128, 128, "bf16", "f32", seed=3)
    assert tv.tv_linear_attn_workspace_size(12, 6428, 600, 16, 128, 128) == 0
    _, S, err = L.prompt(c, max_len=600)
    want = torch.from_numpy(recurrence(c)[1]).to(DEV)
    assert not any(err)
    assert float((S.double() - want).norm() / want.norm()) <= bound(5)


"""fp32 inputs.  A token's product is rounded into the state to nearest, once: mean zero, at most u, so sqrt(T) u
in the norm if every one of T tokens remained.  Its dot products and scalings take a few u more, decays none: they
are products of two floats.  A state to which nothing is added keeps to those few."""


def bound32(tokens, adds=True):
    return (tokens ** 0.5 * U if adds else 0.0) + 2.0 ** -22


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,H,dk,dv", [(8192, 128, 128, 128), (20000, 7, 128, 128), (9001, 7, 64, 64), (300, 7, 64, 128),
                                       (333, 7, 128, 64)])
def test_state_of_fp32_prompts(kind, T, H, dk, dv):
    cut = tv.tv_linear_attn_workspace_size(1, T, T, H, dk, dv, torch.float32) > 0
    assert cut == (H < 128)
    c = make(T, H, dk, dv, kind, torch.float32)
    _, S, err = L.prompt(c)
    assert not any(err)
    k, far = c["k"][:, 0].double(), torch.arange(T - 1, -1, -1, dtype=torch.float64, device=DEV)
    for h in range(7):
        a = c["alpha"][h].double()
        want = (c["v"][:, h].double() * (a ** far)[:, None]).T @ k + c["S0"][0, h].double() * a ** T
        off = float((S[0, h].double() - want).norm() / want.norm().clamp_min(1e-30))
        assert off <= bound32(T, kind not in ("no keys", "no values", "first token")), (h, float(a), off)


def test_fp32_outputs_across_fast_and_slow_blocks():
    # blocks that pass the range of 1 / D between others, resets, decays of 1, a ragged end
    T, H = 1501, 6
    g = torch.Generator().manual_seed(5)
    alpha = torch.rand(T, H, generator=g) ** torch.tensor([0.0, 1e-6, 1e-3, 0.1, 1.0, 8.0])
    alpha[200:216, 1:] = 1e-3
    alpha[640, :4] = 0.0
    alpha[900:1000, 2] = 1.0
    c = L.make([T - 7, 7], 3, H, 128, 128, "f32", "f32", seed=2, alpha=alpha)
    out, S, err = L.prompt(c, max_len=T)
    assert not any(err)
    (o, s), (ao, as_) = recurrence(c), recurrence(c, absolute=True)
    L.check(out, o, ao, T, 128, "f32", "out")
    L.check(S, s, as_, T, 128, "f32", "S")
