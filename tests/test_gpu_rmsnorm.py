"""The gated norm and the residual norm against the fp64 oracle.

Bounds, u = 2^-24: a sum of d squares in fp32, its mean, the root and the products behind one value
are off by at most (d / 2 + 16) u of it (the mean's error halves under the root; the hardware root
and quotient by a few u; the exponential behind the gate by a few u of its argument, |g| < 8); a
residual sum by that of its addend plus u of the result; a norm of it by the same again, relative to
the row's largest addend.  One rounding on a bf16 store: 2^-8 of the value.
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
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(g, *shape, dtype, scale=1.0, shift=0.0):
    return (shift + scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def f64(t):
    return None if t is None else W.f64(t.cpu())


def check(got, want, tol, what):
    g = f64(got)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.isfinite(g).all(), what
    over = np.abs(g - want) - tol
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} of {over.size} past the bound, worst by {over.max():.3e}"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("rows,H,d", [(1, 1, 1), (3, 2, 7), (5, 3, 64), (9, 16, 128), (2, 5, 130), (4, 2, 256),
                                      (3, 2, 257), (2, 1, 1000), (2, 2, 4096), (1, 1, 9001), (2, 1, 32768)])
def test_gated_norm(io, gate_first, rows, H, d):
    g = torch.Generator().manual_seed(d)
    t = TYPES[io]
    x, w = rand(g, rows, H, d, dtype=t, scale=0.3), rand(g, d, dtype=t, scale=0.1)
    gate = rand(g, rows, H * d + 24, dtype=t)[:, 8:8 + H * d].unflatten(1, (H, d))   # a slice
    out = torch.full_like(x, 7.0)
    tv.tv_gated_rmsnorm(x, gate, w, out, EPS, gate_first=gate_first, weight_offset=1.0)
    want = M.gated_rmsnorm(f64(x), f64(gate), f64(w), EPS, gate_first, 1.0)
    check(out, want, (d / 2 + 16) * U * np.abs(want), "out")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("d", [40, 96, 130])
def test_gated_norm_rows_at_any_offset(io, shift, d):
    # x, gate and out start at different places relative to 16 bytes
    g = torch.Generator().manual_seed(shift)
    t = TYPES[io]
    x = rand(g, 5, 2 * d + shift + 1, dtype=t)[:, shift:shift + 2 * d].unflatten(1, (2, d))
    gate = rand(g, 5, 2 * d + 3, dtype=t)[:, 1:1 + 2 * d].unflatten(1, (2, d))
    w = rand(g, d + 1, dtype=t)[1:]
    room = torch.full((5, 2 * d + 9), 7.0, dtype=t, device=DEV)
    out = room[:, 5:5 + 2 * d].unflatten(1, (2, d))
    tv.tv_gated_rmsnorm(x, gate, w, out, EPS)
    want = M.gated_rmsnorm(f64(x), f64(gate), f64(w), EPS)
    check(out, want, (d / 2 + 16) * U * np.abs(want), "out")
    assert bool((room[:, :5] == 7).all()) and bool((room[:, 5 + 2 * d:] == 7).all())


def test_gated_norm_optional_arguments_in_place_and_edges():
    g = torch.Generator().manual_seed(0)
    x = rand(g, 6, 2, 128, dtype=torch.float32)
    want = M.gated_rmsnorm(f64(x), None, None, EPS)
    got = x.clone()
    tv.tv_gated_rmsnorm(got, None, None, got, EPS)              # in place, no gate, no weight
    check(got, want, (64 + 16) * U * np.abs(want), "plain norm")
    empty = x[:0]
    tv.tv_gated_rmsnorm(empty, empty, None, empty.clone(), EPS)
    zero = torch.zeros(2, 1, 128, device=DEV)
    out = torch.full_like(zero, 7.0)
    tv.tv_gated_rmsnorm(zero, torch.ones_like(zero), None, out, EPS)   # a row of zeros stays zero
    torch.cuda.synchronize()
    assert not out.any()
    gate = torch.tensor([-1e4, -90.0, 0.0, 90.0, 1e4], device=DEV).repeat(1, 1, 1)
    ones, out = torch.ones_like(gate), torch.empty_like(gate)
    tv.tv_gated_rmsnorm(ones, gate, None, out, 0.0)             # the gate's far ends
    torch.cuda.synchronize()
    assert out[0, 0, :3].abs().max() < 1e-30 and torch.equal(out[0, 0, 3:].cpu(), torch.tensor([90.0, 1e4]))


TYPE_SETS = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("io,res", TYPE_SETS)
@pytest.mark.parametrize("post,gated,last", [(False, False, False), (True, False, False), (False, True, False),
                                             (True, True, False), (True, True, True)])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 9), (2, 256), (5, 1001), (3, 4096), (2, 5120), (2, 8190), (1, 32768)])
def test_residual_norm(io, res, post, gated, last, rows, D):
    g = torch.Generator().manual_seed(D)
    t, tr = TYPES[io], TYPES[res]
    y = rand(g, rows, D, dtype=t)
    r = rand(g, rows, D + 4, dtype=tr, scale=3.0)[:, 4:]
    pw = rand(g, D, dtype=t, scale=0.1, shift=1.0) if post else None
    w = rand(g, D, dtype=t, scale=0.1, shift=1.0)
    gate = rand(g, rows, D, dtype=t) if gated else None
    ro, out = torch.full((rows, D), 7.0, dtype=tr, device=DEV), torch.full_like(y, 7.0)
    tv.tv_residual_rmsnorm(y, r, ro, EPS, out=None if last else out, weight=w, post_weight=pw, gate=gate, scale=0.7)
    want_r, want = M.residual_rmsnorm(f64(y), f64(r), EPS, f64(w), f64(pw), f64(gate), 0.7)
    add = np.abs(want_r - f64(r))
    tol = (D / 2 + 16) * U * add + 2 * U * np.abs(want_r)
    check(ro, want_r, tol, "residual_out")
    if last:
        assert bool((out == 7).all())
        return
    inv = np.abs(f64(w)) / np.sqrt(np.mean(want_r ** 2, -1, keepdims=True) + EPS)   # |want / want_r|
    check(out, want, inv * tol + (D + 32) * U * np.abs(want), "out")


@pytest.mark.parametrize("io,res", TYPE_SETS)
@pytest.mark.parametrize("D", [511, 2048, 4999])
def test_residual_norm_in_place(io, res, D):
    g = torch.Generator().manual_seed(1)
    y, r = rand(g, 7, D, dtype=TYPES[io]), rand(g, 7, D, dtype=TYPES[res])
    w = rand(g, D, dtype=TYPES[io])
    ro, out = torch.empty_like(r), torch.empty_like(y)
    tv.tv_residual_rmsnorm(y, r, ro, EPS, out=out, weight=w, post_weight=w)
    tv.tv_residual_rmsnorm(y, r, r, EPS, out=y, weight=w, post_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(ro, r) and torch.equal(out, y)


def test_wrong_tensors_are_refused():
    x = torch.zeros(3, 2, 64, device=DEV)
    with pytest.raises(ValueError):
        tv.tv_gated_rmsnorm(x, x[:2], None, x, EPS)
    with pytest.raises(ValueError):
        tv.tv_gated_rmsnorm(x, x, torch.zeros(64, dtype=torch.bfloat16, device=DEV), x, EPS)
    with pytest.raises(ValueError):
        tv.tv_gated_rmsnorm(x.transpose(1, 2), None, None, x, EPS)
    y = torch.zeros(3, 64, device=DEV)
    with pytest.raises(ValueError):
        tv.tv_residual_rmsnorm(y, y, y[:, :32], EPS)
    with pytest.raises(tv.TVError):
        tv.tv_residual_rmsnorm(y, y, y, float("nan"))
    with pytest.raises(tv.TVError):                                # an fp32 block with a bf16 stream
        tv.tv_residual_rmsnorm(y, y.bfloat16(), y.bfloat16(), EPS)
