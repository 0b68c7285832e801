"""Host-side refusals of the windowed attention's, the rotation's and the sampled acceptance's calls (CPU only: no call
here reaches a GPU)."""
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
INF, NAN = float("inf"), float("nan")


def call(name, names, base, **changes):
    return getattr(tv.lib, name)(*[{**base, **changes}[n] for n in names])


ROTATE = ("q qs k ks v vs qw kw cu prefix live B T Hq Hkv hd rotary io norm eps offset theta qo qos ko kos kc vc blocks "
          "table most bs err stream").split()
ROTATE_OK = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, qw=P, kw=P, cu=P, prefix=P, live=P, B=2, T=7, Hq=4, Hkv=2, hd=128,
                 rotary=128, io=tv.TV_BF16, norm=1, eps=1e-6, offset=0.0, theta=1e4, qo=P, qos=512, ko=P, kos=256, kc=P,
                 vc=P, blocks=9, table=P, most=4, bs=16, err=P, stream=None)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(q=None)), (BAD, dict(k=EIGHT)), (BAD, dict(v=None)), (BAD, dict(qw=EIGHT)), (BAD, dict(kw=ODD)),
    (BAD, dict(cu=ODD)), (BAD, dict(cu=None)), (BAD, dict(prefix=None)), (BAD, dict(prefix=ODD)), (BAD, dict(live=ODD)),
    (BAD, dict(B=0)), (BAD, dict(T=-1)), (BAD, dict(Hq=0)), (BAD, dict(Hkv=0)), (NONE, dict(hd=96, rotary=96)),
    (NONE, dict(rotary=24)), (BAD, dict(rotary=144)), (BAD, dict(rotary=-16)), (BAD, dict(io=7)), (NONE, dict(io=tv.TV_F32)),
    (BAD, dict(norm=2)), (BAD, dict(eps=-1.0)), (BAD, dict(eps=NAN)), (BAD, dict(offset=INF)), (BAD, dict(theta=0.5)),
    (BAD, dict(theta=INF)), (BAD, dict(theta=NAN)), (BAD, dict(qs=508)), (BAD, dict(qs=516)), (BAD, dict(ks=248)),
    (BAD, dict(vs=252)), (BAD, dict(qo=None)), (BAD, dict(qos=504)), (BAD, dict(ko=EIGHT)), (BAD, dict(kos=100)),
    (BAD, dict(kc=None)), (BAD, dict(vc=None)), (BAD, dict(kc=EIGHT)), (BAD, dict(blocks=0)), (BAD, dict(table=None)),
    (BAD, dict(most=0)), (NONE, dict(most=(1 << 26) + 1)), (NONE, dict(bs=32)), (BAD, dict(err=None)), (BAD, dict(err=ODD)),
    (BAD, dict(kc=None, vc=None, ko=None)), (NONE, dict(Hq=1 << 17, qs=1 << 24, qos=1 << 24)),
])
def test_rotate_refusals(want, changes):
    assert call("tv_qk_norm_rope", ROTATE, ROTATE_OK, **changes) == want


PROMPT = ("q qs kc vc blocks table most cu prefix B T max_len Hq Hkv hd bs window sinks scale out os ws ws_bytes err "
          "stream").split()
PROMPT_OK = dict(q=P, qs=512, kc=P, vc=P, blocks=9, table=P, most=4, cu=P, prefix=P, B=2, T=7, max_len=7, Hq=4, Hkv=2, hd=128,
                 bs=16, window=5, sinks=1, scale=0.1, out=P, os=512, ws=P, ws_bytes=1 << 40, err=P, stream=None)
COMMON = [
    (BAD, dict(q=None)), (BAD, dict(q=EIGHT)), (BAD, dict(kc=None)), (BAD, dict(vc=EIGHT)), (BAD, dict(blocks=0)),
    (BAD, dict(table=None)), (BAD, dict(table=ODD)), (BAD, dict(most=0)), (NONE, dict(most=(1 << 26) + 1)),
    (BAD, dict(prefix=None)), (BAD, dict(B=0)), (BAD, dict(Hq=5)), (BAD, dict(Hkv=0)), (NONE, dict(hd=96)), (NONE, dict(bs=8)),
    (BAD, dict(window=-1)), (BAD, dict(sinks=-1)), (BAD, dict(scale=NAN)), (BAD, dict(scale=INF)), (BAD, dict(out=None)),
    (BAD, dict(qs=511)), (BAD, dict(qs=516)), (BAD, dict(os=256)), (BAD, dict(err=None)),
    (NONE, dict(Hq=258, qs=1 << 16, os=1 << 16)), (NONE, dict(blocks=1 << 30)), (NONE, dict(B=1 << 24)), (NONE, dict(Hq=1 << 17, Hkv=1 << 17, qs=1 << 25, os=1 << 25)),
]


@cpu_only
@pytest.mark.parametrize("want,changes", COMMON + [(BAD, dict(cu=None)), (BAD, dict(cu=ODD)), (BAD, dict(T=-1)),
                                                   (BAD, dict(max_len=-1))])
def test_prompt_refusals(want, changes):
    assert call("tv_window_attn_prompt", PROMPT, PROMPT_OK, **changes) == want


STEP = "q qs kc vc blocks table most prefix live B Hq Hkv hd bs window sinks scale out os ws ws_bytes err stream".split()
STEP_OK = {n: PROMPT_OK.get(n) for n in STEP} | dict(live=P)


@cpu_only
@pytest.mark.parametrize("want,changes", COMMON + [(BAD, dict(live=ODD))])
def test_step_refusals(want, changes):
    assert call("tv_window_attn_step", STEP, STEP_OK, **changes) == want


SAMPLE = "parents tokens target draft uniforms B N V Lmax probs path length next err stream".split()
SAMPLE_OK = dict(parents=P, tokens=P, target=P, draft=P, uniforms=P, B=2, N=5, V=100, Lmax=5, probs=tv.TV_F32, path=P, length=P,
                 next=P, err=P, stream=None)


@cpu_only
@pytest.mark.parametrize("want,changes", [
    (BAD, dict(parents=None)), (BAD, dict(tokens=ODD)), (BAD, dict(target=None)), (BAD, dict(target=EIGHT)),
    (BAD, dict(draft=EIGHT)), (BAD, dict(uniforms=None)), (BAD, dict(B=0)), (BAD, dict(N=0)), (BAD, dict(V=0)),
    (BAD, dict(Lmax=0)), (BAD, dict(probs=3)), (BAD, dict(path=None)), (BAD, dict(length=ODD)), (BAD, dict(next=None)),
    (BAD, dict(err=None)), (NONE, dict(N=257)), (NONE, dict(V=(1 << 24) + 1)), (NONE, dict(B=(1 << 24) + 1)),
])
def test_sample_refusals(want, changes):
    assert call("tv_accept_sample", SAMPLE, SAMPLE_OK, **changes) == want


def test_workspace_size_is_host_only():
    size = tv.tv_window_attn_workspace_size
    assert size(0, 8, 8, 4, 2, 128, 4) == 0 and size(1, 8, 8, 4, 2, 96, 4) == 0 and size(1, 8, 8, 5, 2, 128, 4) == 0
    assert size(1, 8, 8, 4, 2, 128, 4) == size(1, 8, 100, 4, 2, 128, 4)      # max_len past T
    assert size(1, 0, 0, 4, 2, 128, 4) == 0


def test_the_binding_refuses_host_tensors():
    q, k, n, bf = torch.zeros(2, 4, 128), torch.zeros(2, 2, 128), torch.zeros(2, dtype=torch.int32), torch.bfloat16
    cache, table = torch.zeros(3, 2, 16, 128, dtype=bf), torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        tv.tv_qk_norm_rope(q, k, q, n, n, k_out=k)
    with pytest.raises(ValueError):
        tv.tv_qk_norm_rope(q.half(), k.half(), q.half(), n, n, k_out=k.half())
    with pytest.raises(ValueError):
        tv.tv_window_attn_step(q.to(bf), cache, cache, table, n, q.to(bf), n)
    with pytest.raises(ValueError):
        tv.tv_accept_sample(table, table, torch.zeros(2, 1, 5), None, torch.zeros(2, 1), table, n, n, n)


def test_status_string():
    assert "probability" in tv.status_string(tv.TV_ERR_BAD_PROBS) and tv.TV_ERR_BAD_PROBS == -11
