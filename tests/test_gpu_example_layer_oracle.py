"""The linear-attention layer of ``examples/`` against the layer in 64 bits.

bf16 values between the calls: the projection, the mixer's output, the gated norm, the block's output and
the next norm, each rounded once, at most half a step, u = 2^-8 of a value, uniform within it: u / sqrt(3) in
the norm.  The projection's roundings reach the output by three ways at once (keys, queries and values multiply;
the gate by one more), each by a factor of order one; the others by one: sqrt(4 + 4) u / sqrt(3) if independent, and
twice that is allowed.  The residual stream itself is fp32 and takes the block's output only: no more.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import workloads as W
from oracle import mixer as M

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"
TOL = 2 * 8 ** 0.5 * 2.0 ** -8 / 3 ** 0.5


def _layer(*args):
    spec = importlib.util.spec_from_file_location("linear_attention_layer_o",
                                                  os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod.Layer(*args), mod.EPS


def f64(t):
    return W.f64(t.cpu())


def in_64_bits(layer, eps, x, residual, cu, S0):
    q, k, v, z, a, _ = np.split(f64(x) @ f64(layer.w_in), np.cumsum(layer.split)[:-1], axis=1)
    T = len(q)
    alpha = 1 / (1 + np.exp(-(a + 3)))
    q, k = q.reshape(T, layer.Hk, layer.dk), k.reshape(T, layer.Hk, layer.dk)
    v, z = v.reshape(T, layer.H, layer.dv), z.reshape(T, layer.H, layer.dv)
    o, S = M.linear_attn(q, k, v, alpha, cu, S0, layer.dk ** -0.5)
    y = M.gated_rmsnorm(o, z, f64(layer.n_head), eps).reshape(T, -1) @ f64(layer.w_out)
    return M.residual_rmsnorm(y, f64(residual), eps, f64(layer.n_next)) + (S,)


def off(got, want):
    return np.linalg.norm(f64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("sizes", [(512, 8, 4, 128, 128), (256, 4, 4, 64, 64)])
def test_layer(sizes):
    layer, eps = _layer(*sizes)
    g = torch.Generator(device=DEV).manual_seed(3)
    lens = [300, 1, 77]
    T, cu = sum(lens), [0, 300, 301, 378]
    x = torch.randn(T, sizes[0], generator=g, device=DEV).bfloat16()
    S = torch.empty(3, layer.H, layer.dv, layer.dk, device=DEV)
    (r, nxt), err = layer.prompts(x, x.float(), torch.tensor(cu, dtype=torch.int32, device=DEV), 300, S)
    want_r, want_x, want_S = in_64_bits(layer, eps, x, x.float(), cu, None)
    assert not err.any()
    add = want_r - f64(x)
    assert np.linalg.norm(f64(r) - want_r) <= TOL * np.linalg.norm(add)
    assert off(nxt, want_x) <= TOL and off(S, want_S) <= TOL
    x = torch.randn(3, sizes[0], generator=g, device=DEV).bfloat16()
    r, nxt = layer.token(x, x.float(), S)
    want_r, want_x, want_S = in_64_bits(layer, eps, x, x.float(), [0, 1, 2, 3], want_S)
    assert np.linalg.norm(f64(r) - want_r) <= TOL * np.linalg.norm(want_r - f64(x))
    assert off(nxt, want_x) <= TOL and off(S, want_S) <= TOL
