"""Rotation at far positions, up to the last one, against angles of 80 decimal digits.

An angle is good to 2^-27 of a turn at every position, and a cosine or sine of it to 2 ulp of a number below 1, 2^-23: so
a pair (1, 0) turns to within 2 pi 2^-27 + 2^-23 of it.  With norms and weights the bound is that of near positions, 32 u
(|a| + |b|) of a pair, u = 2^-24: 25 u of it are used there, 1 u by this angle."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import DEV, U, f64, whole
from oracle import window as O

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
STARTS = [0, 131071, (1 << 24) + 1, 10 ** 9, (1 << 30) - 5, (1 << 31) - 4]     # three tokens each: 2^31 - 2 is the last place
LENS = [3] * len(STARTS)
AT = [p + i for p in STARTS for i in range(3)]


def cos_sin(positions, rotary, theta):
    """[positions, rotary / 2] in 64 bits."""
    cs = np.zeros((2, len(positions), rotary // 2))
    with localcontext() as ctx:
        ctx.prec = 80
        for c in range(rotary // 2):
            turn = Decimal(theta) ** (Decimal(-2 * c) / Decimal(rotary)) / (2 * PI)
            for i, p in enumerate(positions):
                a = 2 * math.pi * float(p * turn % 1)
                cs[:, i, c] = math.cos(a), math.sin(a)
    return cs


def rotate(q, k, rotary, theta, cu, **more):
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    starts, B = (STARTS, len(STARTS)) if cu else (AT, len(AT))
    err = torch.full((B,), 9, dtype=torch.int32, device=DEV)
    tv.tv_qk_norm_rope(q, k, q_out, whole(starts), err, k_out=k_out, cu_seqlens=whole(np.cumsum([0] + LENS)) if cu else None,
                       rotary_dim=rotary, rope_theta=theta, **more)
    torch.cuda.synchronize()
    assert not err.any()
    return f64(q_out), f64(k_out)


@pytest.mark.parametrize("cu", [True, False])
@pytest.mark.parametrize("hd,rotary", [(64, 64), (128, 112), (256, 256)])
@pytest.mark.parametrize("theta", [1.0, 1e4, 1e7])
def test_angles(theta, hd, rotary, cu):
    x = torch.zeros(len(AT), 1, hd, device=DEV)
    x[..., :rotary // 2] = 1.0
    want = cos_sin(AT, rotary, theta)
    for got in rotate(x, x.clone(), rotary, theta, cu, norm=False):
        for part, w in zip((got[:, 0, :rotary // 2], got[:, 0, rotary // 2:rotary]), want):
            off = np.abs(part - w)
            assert off.max() <= 2 * math.pi * 2.0 ** -27 + 2.0 ** -23, (off.max(), np.argwhere(off == off.max()))
        assert (got[..., rotary:] == 0).all()


@pytest.mark.parametrize("theta", [1.0, 1e4, 1e7])
def test_norms_weights_and_rotation(theta):
    g = torch.Generator().manual_seed(3)
    q, k = (torch.randn(len(AT), n, 128, generator=g).to(DEV) for n in (2, 1))
    w = (1 + 0.2 * torch.randn(128, generator=g)).to(DEV)
    cos, sin = cos_sin(AT, 128, theta)[:, :, None]
    for x, got in zip((q, k), rotate(q, k, 128, theta, True, q_weight=w, k_weight=w, eps=1e-6)):
        y = O.norm_rotate(f64(x), f64(w), AT, 0, theta, 1e-6)
        a, b = y[..., :64], y[..., 64:]
        want = np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)
        size = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
        assert (np.abs(got - want) <= 32 * U * size).all()
