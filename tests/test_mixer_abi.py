"""Host-side refusals of the linear-attention and norm calls (CPU only: no call here reaches a GPU)."""
import ctypes

import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-address stand-ins; CPU only")
BAD, NONE = tv.TV_ERR_INVALID_ARG, tv.TV_ERR_UNSUPPORTED
BUF = ctypes.create_string_buffer(4096)
P = ctypes.c_void_p((ctypes.addressof(BUF) + 255) & ~255)
ODD = ctypes.c_void_p(P.value + 1)
EIGHT = ctypes.c_void_p(P.value + 8)


def call(name, names, base, **changes):
    return getattr(tv.lib, name)(*[{**base, **changes}[n] for n in names])


PROMPT = ("q qs k ks v vs alpha as_ S0 cu B T max_len Hk H dk dv io state q_scale out os S ws ws_bytes err stream").split()
PROMPT_OK = dict(q=P, qs=256, k=P, ks=256, v=P, vs=512, alpha=P, as_=4, S0=P, cu=P, B=2, T=64, max_len=64, Hk=2, H=4,
                 dk=128, dv=128, io=tv.TV_BF16, state=tv.TV_BF16, q_scale=1.0, out=P, os=512, S=P, ws=None, ws_bytes=0,
                 err=P, stream=None)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(q=None)), (BAD, dict(k=EIGHT)), (BAD, dict(v=ODD)), (BAD, dict(alpha=None)), (BAD, dict(S0=EIGHT)),
    (BAD, dict(cu=None)), (BAD, dict(out=None)), (BAD, dict(S=None)), (BAD, dict(err=None)), (BAD, dict(B=0)),
    (BAD, dict(T=-1)), (BAD, dict(max_len=-1)), (BAD, dict(H=3)), (BAD, dict(Hk=0)), (NONE, dict(dk=96)),
    (NONE, dict(dv=32)), (BAD, dict(io=5)), (NONE, dict(io=tv.TV_F32)), (BAD, dict(q_scale=float("inf"))),
    (BAD, dict(qs=248)), (BAD, dict(ks=260)), (BAD, dict(vs=504)), (BAD, dict(os=516)), (BAD, dict(as_=3)),
    (BAD, dict(as_=-4)), (NONE, dict(B=1 << 25)),
])
def test_prompt_refusals(want, changes):
    assert call("tv_linear_attn_prompt", PROMPT, PROMPT_OK, **changes) == want


@cpu_only
def test_prompt_needs_its_workspace():
    big = dict(B=1, T=1 << 20, max_len=1 << 20)
    need = tv.tv_linear_attn_workspace_size(1, 1 << 20, 1 << 20, 4, 128, 128)
    assert need > 0
    assert call("tv_linear_attn_prompt", PROMPT, PROMPT_OK, **big) == BAD
    assert call("tv_linear_attn_prompt", PROMPT, PROMPT_OK, **big, ws=P, ws_bytes=need - 1) == BAD
    assert call("tv_linear_attn_prompt", PROMPT, PROMPT_OK, **big, ws=EIGHT, ws_bytes=need) == BAD


def test_workspace_size_is_host_only():
    size = tv.tv_linear_attn_workspace_size
    assert size(64, 64 * 100, 100, 32, 128, 128) == 0          # many short prompts: none is cut
    assert size(1, 0, 0, 4, 128, 128) == 0 and size(0, 8, 8, 4, 128, 128) == 0 and size(1, 8, 8, 4, 96, 128) == 0
    assert size(1, 1 << 16, 1 << 16, 4, 128, 128) == size(1, 1 << 16, 1 << 20, 4, 128, 128)   # max_len past T


STEP = "q qs k ks v vs alpha as_ live B Hk H dk dv io state q_scale out os S stream".split()
STEP_OK = {n: PROMPT_OK.get(n) for n in STEP} | dict(live=P)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(q=None)), (BAD, dict(k=None)), (BAD, dict(v=EIGHT)), (BAD, dict(alpha=ODD)), (BAD, dict(live=ODD)),
    (BAD, dict(B=0)), (BAD, dict(H=5)), (NONE, dict(dk=32)), (NONE, dict(io=tv.TV_F32)), (BAD, dict(state=9)),
    (BAD, dict(out=None)), (BAD, dict(S=EIGHT)), (BAD, dict(os=100)), (BAD, dict(q_scale=float("nan"))),
    (BAD, dict(vs=513)),
])
def test_step_refusals(want, changes):
    assert call("tv_linear_attn_step", STEP, STEP_OK, **changes) == want


GATED = "x xs gate gs weight rows H d io eps offset first out os stream".split()
GATED_OK = dict(x=P, xs=256, gate=P, gs=256, weight=P, rows=3, H=2, d=128, io=tv.TV_BF16, eps=1e-6, offset=0.0, first=0,
                out=P, os=256, stream=None)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(x=None)), (BAD, dict(x=ODD)), (BAD, dict(gate=ODD)), (BAD, dict(weight=ODD)), (BAD, dict(out=None)),
    (BAD, dict(xs=255)), (BAD, dict(gs=255)), (BAD, dict(os=255)), (BAD, dict(rows=-1)), (BAD, dict(H=0)), (BAD, dict(d=0)),
    (NONE, dict(d=32769, xs=1 << 20, gs=1 << 20, os=1 << 20)), (BAD, dict(io=2)), (BAD, dict(eps=-1.0)),
    (BAD, dict(eps=float("nan"))), (BAD, dict(offset=float("inf"))), (BAD, dict(first=2)),
    (NONE, dict(rows=1 << 30, H=2)), (NONE, dict(rows=(1 << 31) - 1, H=1, xs=1 << 20)), (tv.TV_OK, dict(rows=0, x=None)),
])
def test_gated_norm_refusals(want, changes):
    assert call("tv_gated_rmsnorm", GATED, GATED_OK, **changes) == want


RES = "y ys r rs pw gate gs scale w rows D io res eps offset ro ros out os stream".split()
RES_OK = dict(y=P, ys=64, r=P, rs=64, pw=P, gate=P, gs=64, scale=1.0, w=P, rows=3, D=64, io=tv.TV_BF16, res=tv.TV_F32,
              eps=1e-6, offset=0.0, ro=P, ros=64, out=P, os=64, stream=None)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(y=None)), (BAD, dict(r=None)), (BAD, dict(r=ctypes.c_void_p(P.value + 2))), (BAD, dict(pw=ODD)),
    (BAD, dict(gate=ODD)), (BAD, dict(w=ODD)), (BAD, dict(ro=None)), (BAD, dict(out=ODD)), (BAD, dict(ys=63)),
    (BAD, dict(rs=63)), (BAD, dict(gs=63)), (BAD, dict(ros=63)), (BAD, dict(os=63)), (BAD, dict(D=0)), (BAD, dict(rows=-1)),
    (NONE, dict(D=32769)), (NONE, dict(io=tv.TV_F32, res=tv.TV_BF16)), (BAD, dict(io=3)), (BAD, dict(scale=float("inf"))),
    (BAD, dict(eps=float("inf"))), (tv.TV_OK, dict(rows=0)),
])
def test_residual_norm_refusals(want, changes):
    assert call("tv_residual_rmsnorm", RES, RES_OK, **changes) == want


def test_status_string():
    assert "cu_seqlens" in tv.status_string(tv.TV_ERR_BAD_SEQLEN)
