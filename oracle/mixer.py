"""Linear attention with a decay, and the norms around a mixer, in fp64.

Plain loops over the definitions: the recurrence token by token, every norm from its formula.
"""
from __future__ import annotations

import numpy as np


def linear_attn(q, k, v, alpha, cu_seqlens, S0=None, q_scale: float = 1.0):
    """q, k [T, Hk, dk], v [T, H, dv], alpha [T, H] or [H]; S0 [B, H, dv, dk] or None (zero).
    S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = S_t (q_scale q_t).  Returns o [T, H, dv] (zero where
    no prompt has a token) and the final states."""
    q, k, v, alpha = (np.asarray(x, dtype=np.float64) for x in (q, k, v, alpha))
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    alpha = np.broadcast_to(alpha, (T, H))
    B = len(cu_seqlens) - 1
    S = np.zeros((B, H, dv, dk)) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((T, H, dv))
    head = np.arange(H) // (H // Hk)
    for b in range(B):
        for t in range(int(cu_seqlens[b]), int(cu_seqlens[b + 1])):
            S[b] = alpha[t][:, None, None] * S[b] + v[t][:, :, None] * k[t, head][:, None, :]
            o[t] = np.einsum("hvk,hk->hv", S[b], q_scale * q[t, head])
    return o, S


def silu(g):
    g = np.asarray(g, dtype=np.float64)
    return g / (1.0 + np.exp(-g))


def rmsnorm(x, eps: float, weight=None, weight_offset: float = 0.0):
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return n if weight is None else n * (weight_offset + np.asarray(weight, dtype=np.float64))


def gated_rmsnorm(x, gate, weight, eps: float, gate_first: bool = False, weight_offset: float = 0.0):
    g = 1.0 if gate is None else silu(gate)
    x = np.asarray(x, dtype=np.float64)
    if gate_first:
        return rmsnorm(x * g, eps, weight, weight_offset)
    return rmsnorm(x, eps, weight, weight_offset) * g


def residual_rmsnorm(y, residual, eps: float, weight=None, post_weight=None, gate=None, scale: float = 1.0,
                     weight_offset: float = 0.0):
    """(residual + scale * gate * post-norm(y), its norm)."""
    t = np.asarray(y, dtype=np.float64)
    if post_weight is not None:
        t = rmsnorm(t, eps, post_weight, weight_offset)
    if gate is not None:
        t = np.asarray(gate, dtype=np.float64) * t
    r = np.asarray(residual, dtype=np.float64) + scale * t
    return r, rmsnorm(r, eps, weight, weight_offset)
