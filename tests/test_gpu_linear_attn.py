"""Linear attention with a decay against the fp64 oracle: whole prompts and single tokens.

Bounds, per element, from the oracle run on absolute values (A = the sum of |terms| behind the
element), u = 2^-24 (half an fp32 step):
  * a sum of n tokens, each scaled by up to n decays, and a dot product over dk columns in fp32:
    (2 n + dk + 8) u A;
  * bf16 inputs may go through the matrix units, where scores, decayed keys and states enter as a
    bf16 value and a bf16 remainder (2^-16 of the operand left out, three operands) and decays as
    powers of two of rounded logarithms (exponents below 150 that matter: 2^-16): 2^-14 A;
  * a result stored in bf16 is rounded once: 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
import workloads as W
from oracle import mixer as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lens, Hk, H, dk, dv, io="bf16", state="bf16", seed=0, per_head=False, fused=True, alpha=None):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lens), len(lens)
    q, k, v = (torch.randn(T, n, d, generator=g) for n, d in ((Hk, dk), (Hk, dk), (H, dv)))
    q, k = torch.nn.functional.normalize(q, dim=-1), torch.nn.functional.normalize(k, dim=-1)
    if alpha is None:
        span = 2.0 ** -torch.linspace(0, 11, H)
        alpha = 1 - span / 2 if per_head else torch.exp(-torch.nn.functional.softplus(torch.randn(T, H, generator=g)) * span)
    whole = torch.cat([x.flatten(1) for x in (q, k, v)], 1).to(TYPES[io]).to(DEV)
    parts = whole.split([Hk * dk, Hk * dk, H * dv], dim=1)
    q, k, v = (x.unflatten(1, s) for x, s in zip(parts, ((Hk, dk), (Hk, dk), (H, dv))))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    S0 = (0.1 * torch.randn(B, H, dv, dk, generator=g)).to(TYPES[state]).to(DEV)
    return dict(q=q, k=k, v=v, alpha=alpha.float().to(DEV), cu=cu.to(DEV), S0=S0)


def prompt(c, S0="S0", in_place=False, max_len=None, q_scale=0.5, workspace=None, stream=None):
    T, H, dv = c["v"].shape
    B = c["cu"].numel() - 1
    out = torch.full((T, H, dv), 7.0, dtype=c["v"].dtype, device=DEV)
    S0 = None if S0 is None else c["S0"].clone()
    S = S0 if in_place else torch.full_like(c["S0"], 7.0)
    err = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    tv.tv_linear_attn_prompt(c["q"], c["k"], c["v"], c["alpha"], c["cu"], out, S, err, S0=S0, max_len=max_len,
                             q_scale=q_scale, workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return out, S, err.tolist()


def f64(t):
    return W.f64(t.cpu())


def check(got, want, size, n, dk, io, what):
    tol = ((2 * n + dk + 8) * U + (2.0 ** -14 if io == "bf16" else 0.0)) * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    g = f64(got)
    assert np.isfinite(g).all(), what
    over = np.abs(g - want) - tol
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} of {over.size} past the bound, worst by {over.max():.3e}"


def check_prompt(c, out, S, err, S0=True, q_scale=0.5):
    assert not any(err)
    args = [f64(c[n]) for n in ("q", "k", "v", "alpha")]
    cu = c["cu"].tolist()
    start = f64(c["S0"]) if S0 else None
    o, s = M.linear_attn(*args, cu, start, q_scale)
    ao, as_ = M.linear_attn(*[np.abs(x) for x in args], cu, None if start is None else np.abs(start), q_scale)
    n, dk = max(np.diff(cu)), args[0].shape[-1]
    io = "bf16" if c["v"].dtype == torch.bfloat16 else "f32"
    check(out, o, ao, n, dk, io, "out")
    check(S, s, as_, n, dk, io, "S")


TYPE_SETS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("io,state", TYPE_SETS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_prompt_types_and_head_sizes(io, state, dk, dv):
    c = make([37, 0, 1, 130], 2, 4, dk, dv, io, state, seed=dk + dv)
    check_prompt(c, *prompt(c))


@pytest.mark.parametrize("io,state", TYPE_SETS)
@pytest.mark.parametrize("lens", [[1], [2, 15, 16, 17], [127, 128, 129], [255, 256, 257], [0, 0, 3], [5, 0], [640]])
def test_prompt_lengths(io, state, lens):
    c = make(lens, 3, 3, 128, 128, io, state, seed=sum(lens), per_head=len(lens) == 1)
    check_prompt(c, *prompt(c, S0=None), S0=False)


@pytest.mark.parametrize("io,state", TYPE_SETS)
def test_long_prompt_on_few_heads(io, state):
    # far more tokens than heads: the prompt is cut into segments; the shorter ones are not
    c = make([5003, 70, 0, 1200], 1, 2, 128, 128, io, state, seed=5)
    out, S, err = prompt(c, max_len=5003)
    check_prompt(c, out, S, err)
    again, S2, _ = prompt(c, in_place=True, max_len=5003)
    assert torch.equal(out, again) and torch.equal(S, S2)      # S may be S0 itself, cut or not
    c = make([4097], 2, 2, 64, 64, io, state, seed=6, fused=False)
    check_prompt(c, *prompt(c, S0=None), S0=False)


@pytest.mark.parametrize("lens,H", [([4096], 16), ([1500, 900, 0, 600], 12)])
def test_fewer_segments_than_the_host_can_bound(lens, H):
    # the launch is sized by B + T / segment; the CTAs past the real segments find nothing to do
    c = make(lens, H, H, 64, 64, "bf16", "f32", seed=sum(lens))
    check_prompt(c, *prompt(c, S0=None), S0=False)


def test_prompt_in_place_many_heads():
    c = make([300, 41], 16, 32, 128, 128, seed=8)
    out, S, err = prompt(c)
    check_prompt(c, out, S, err)
    again, S2, _ = prompt(c, in_place=True)
    assert torch.equal(out, again) and torch.equal(S, S2)


@pytest.mark.parametrize("io,state", TYPE_SETS)
def test_prompt_decays_from_zero_to_one(io, state):
    # alpha 0 forgets the state, alpha 1 keeps it; fast decays pass the range of fp32 in a chunk
    T = 300
    g = torch.Generator().manual_seed(1)
    alpha = torch.stack([torch.ones(T), torch.zeros(T), (torch.rand(T, generator=g) < 0.9).float(),
                         torch.full((T,), 1e-3), torch.full((T,), 1e-38), torch.rand(T, generator=g)], 1)
    c = make([T], 6, 6, 128, 128, io, state, seed=2, alpha=alpha)
    check_prompt(c, *prompt(c))


def test_prompt_reset_then_slow_decay_keeps_its_precision():
    # the exponents after a reset are small differences of large sums
    T = 256
    alpha = torch.full((T, 2), 0.999)
    alpha[5:60] = 1e-30
    c = make([T], 2, 2, 128, 128, "bf16", "f32", seed=3, alpha=alpha)
    check_prompt(c, *prompt(c))


@pytest.mark.parametrize("io,state", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_tokens_masked_by_a_zero_key_leave_the_state(io, state):
    c = make([700, 5000], 2, 4, 128, 128, io, state, seed=8, alpha=torch.ones(5700, 4))
    c["k"].zero_()
    _, S, err = prompt(c)
    assert not any(err)
    assert torch.equal(S, c["S0"])


def test_long_prompt_with_a_slow_decay_keeps_an_fp32_state():
    """Every head walks its 64 chunks by itself.  A pair of bf16 leaves half of 2^-16 of a key; the sixteen
    cuts of a pair's products are half a unit of 2^-23 / 1.39 each, and with four units given back at most
    1.8 remain for each chunk that the state has come through.  (A third part leaves less of either.)"""
    T, H, d = 8192, 152, 64
    c = make([T], 8, H, d, d, "bf16", "f32", seed=9, alpha=torch.full((T, H), 0.9999))
    _, S, err = prompt(c)
    assert not any(err)
    a = float(torch.tensor(0.9999).double())  # the decay the kernel gets
    w = a ** torch.arange(T - 1, -1, -1, dtype=torch.float64, device=DEV)
    for h in (0, 77, 151):
        want = (c["v"][:, h].double() * w[:, None]).T @ c["k"][:, h // 19].double() + c["S0"][0, h].double() * a ** T
        off = float((S[0, h].double() - want).norm() / want.norm())
        assert off <= 2.0 ** -17 + 64 * 1.8 * 2.0 ** -23, (h, off)


def test_other_prompts_rows_and_gaps_are_not_touched():
    # NaN and infinity in the next prompt's first tokens, in the rows before the first prompt and
    # behind the last one, reach nobody else
    c = make([9, 150, 100, 61, 8], 2, 2, 128, 128, "bf16", "f32", seed=4)
    cu = c["cu"].clone()
    c["cu"] = cu[1:-1].clone()
    c["S0"] = c["S0"][1:-1].clone()
    keep = {n: c[n].clone() for n in ("q", "k", "v", "alpha")}
    clean, S, err = prompt(c)
    for n in ("q", "k", "v", "alpha"):
        c[n][:9] = float("nan")
        c[n][-8:] = float("inf")
        c[n][9 + 150:9 + 150 + 100] = float("nan")
    out, S2, err2 = prompt(c)
    assert err == err2 == [0, 0, 0]
    rows = list(range(9, 159)) + list(range(259, 320))
    assert torch.equal(out[rows], clean[rows]) and torch.equal(S2[[0, 2]], S[[0, 2]])
    assert bool((out[:9] == 7).all()) and bool((out[-8:] == 7).all())      # rows of no prompt
    c.update(keep)
    check_prompt_rows = [x for x in (out, S2)]
    assert all(torch.isfinite(x[[0, 2]].float()).all() for x in check_prompt_rows[1:])


@pytest.mark.parametrize("cu", [[0, 5, 4], [-1, 3, 6], [0, 3, 7], [0, 6, 6]])
def test_bad_seqlens_write_nothing(cu):
    c = make([3, 3], 1, 2, 128, 128, "bf16", "f32")
    c["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, S, err = prompt(c, max_len=5)
    assert err == [tv.TV_ERR_BAD_SEQLEN] * 2
    assert bool((out == 7).all()) and bool((S == 7).all())


def test_prompt_without_tokens_copies_the_states():
    c = make([4], 1, 2, 64, 64, "bf16", "f32")
    c = dict(c, q=c["q"][:0], k=c["k"][:0], v=c["v"][:0], alpha=c["alpha"][:0],
             cu=torch.zeros(2, dtype=torch.int32, device=DEV))
    out, S, err = prompt(c)
    assert err == [0] and torch.equal(S, c["S0"])
    out, S, err = prompt(c, S0=None)
    assert err == [0] and not S.any()


def test_prompt_on_another_stream_and_with_a_callers_workspace():
    c = make([3000], 2, 2, 128, 128, "bf16", "f32", seed=11)
    want, S, _ = prompt(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    need = tv.tv_linear_attn_workspace_size(1, 3000, 3000, 2, 128, 128)
    ws = torch.full((max(need, 1) + 64,), 0xff, dtype=torch.uint8, device=DEV)   # contents are ignored
    got, S2, err = prompt(c, workspace=ws, stream=side)
    assert err == [0] and torch.equal(got, want) and torch.equal(S, S2)
    assert bool((ws[need:] == 0xff).all())


def test_prompt_in_a_graph():
    c = make([500, 900], 2, 4, 128, 128, seed=12)
    want, S, _ = prompt(c)
    out, S1 = torch.zeros_like(want), torch.zeros_like(S)
    err = torch.zeros(2, dtype=torch.int32, device=DEV)
    need = tv.tv_linear_attn_workspace_size(2, 1400, 1400, 4, 128, 128)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.tv_linear_attn_prompt(c["q"], c["k"], c["v"], c["alpha"], c["cu"], out, S1, err, S0=c["S0"], q_scale=0.5,
                                 workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(S1, S)


# ------------------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("io,state", TYPE_SETS)
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,Hk,H", [(1, 1, 1), (3, 2, 4), (33, 8, 16)])
def test_step(io, state, dk, dv, B, Hk, H):
    c = make([1] * B, Hk, H, dk, dv, io, state, seed=B + dk, per_head=B == 3)
    live = torch.ones(B, dtype=torch.int32, device=DEV)
    live[B // 2] = 0 if B > 1 else 1
    S, out = c["S0"].clone(), torch.full((B, H, dv), 7.0, dtype=c["v"].dtype, device=DEV)
    tv.tv_linear_attn_step(c["q"], c["k"], c["v"], c["alpha"], S, out, live=live, q_scale=0.5)
    torch.cuda.synchronize()
    on = live.bool().cpu()
    assert torch.equal(S[~on.to(DEV)], c["S0"][~on.to(DEV)]) and bool((out[~on.to(DEV)] == 7).all())
    args = [f64(c[n]) for n in ("q", "k", "v", "alpha")]
    o, s = M.linear_attn(*args, list(range(B + 1)), f64(c["S0"]), 0.5)
    ao, as_ = M.linear_attn(*[np.abs(x) for x in args], list(range(B + 1)), np.abs(f64(c["S0"])), 0.5)
    on = on.numpy()
    check(out[live.bool()], o[on], ao[on], 1, dk, "f32", "out")   # no matrix units here
    check(S[live.bool()], s[on], as_[on], 1, dk, "f32", "S")


def test_steps_continue_a_prompt():
    # a prompt, then its next tokens one by one, is the longer prompt
    c = make([140], 2, 4, 128, 128, "f32", "f32", seed=21)
    whole, end, _ = prompt(c)
    head = {n: (c[n][:133] if n in ("q", "k", "v", "alpha") else c[n]) for n in c}
    head["cu"] = torch.tensor([0, 133], dtype=torch.int32, device=DEV)
    first, S, _ = prompt(head)
    out = [first]
    for t in range(133, 140):
        o = torch.empty(1, 4, 128, device=DEV)
        tv.tv_linear_attn_step(c["q"][t:t + 1], c["k"][t:t + 1], c["v"][t:t + 1], c["alpha"][t:t + 1], S, o, q_scale=0.5)
        out.append(o)
    torch.cuda.synchronize()
    args = [np.abs(f64(c[n])) for n in ("q", "k", "v", "alpha")]
    ao, as_ = M.linear_attn(*args, [0, 140], np.abs(f64(c["S0"])), 0.5)
    check(torch.cat(out), f64(whole), 2 * ao, 140, 128, "f32", "out")
    check(S, f64(end), 2 * as_, 140, 128, "f32", "S")


def test_wrong_tensors_are_refused():
    c = make([8], 2, 4, 128, 128)
    out, S, err = torch.empty(8, 4, 128, dtype=torch.bfloat16, device=DEV), c["S0"].clone(), torch.zeros(
        1, dtype=torch.int32, device=DEV)
    args = [c["q"], c["k"], c["v"], c["alpha"], c["cu"], out, S, err]
    for i, bad in ((0, c["q"].float()), (1, c["k"][:7]), (3, c["alpha"].double()), (4, c["cu"].long()),
                   (5, out[:, :2]), (6, S[:, :2]), (0, c["q"].transpose(0, 1))):
        with pytest.raises(ValueError):
            tv.tv_linear_attn_prompt(*[bad if j == i else a for j, a in enumerate(args)])
    with pytest.raises(tv.TVError) as e:          # a workspace that is too small
        long = make([6000], 1, 1, 128, 128, seed=1)
        o = torch.empty(6000, 1, 128, dtype=torch.bfloat16, device=DEV)
        assert tv.tv_linear_attn_workspace_size(1, 6000, 6000, 1, 128, 128) > 16
        tv.tv_linear_attn_prompt(long["q"], long["k"], long["v"], long["alpha"], long["cu"], o, long["S0"].clone(), err,
                                 workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == tv.TV_ERR_INVALID_ARG
