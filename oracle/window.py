"""Windowed softmax attention over a paged cache, the norms and rotation before it, and acceptance by
probabilities, in fp64.

Plain loops over the definitions: a query at a time, a token at a time.
"""
from __future__ import annotations

import numpy as np

from .mixer import rmsnorm

PAGE = 16


def rotate(x, position, rotary: int, theta: float):
    """The first ``rotary`` columns of x [..., hd]: pairs (c, c + rotary/2) turned by position * theta^(-2c/rotary)."""
    x = np.array(x, dtype=np.float64)
    half = rotary // 2
    angle = np.asarray(position, dtype=np.float64)[..., None] * float(theta) ** (-2.0 * np.arange(half) / max(rotary, 1))
    c, s = np.cos(angle), np.sin(angle)
    a, b = x[..., :half].copy(), x[..., half:rotary].copy()
    x[..., :half], x[..., half:rotary] = a * c - b * s, b * c + a * s
    return x


def norm_rotate(x, weight, positions, rotary: int, theta: float, eps: float, norm: bool = True, weight_offset: float = 0.0):
    """x [T, H, hd] at positions [T]."""
    x = np.asarray(x, dtype=np.float64)
    y = rmsnorm(x, eps, weight, weight_offset) if norm else x
    return rotate(y, np.asarray(positions)[:, None], rotary, theta)


def visible(p: int, window: int, sinks: int):
    """Positions of the keys that the query at position p sees."""
    j = np.arange(p + 1)
    return j if window == 0 else j[(p - j < window) | (j < sinks)]


def rows(cache, table_row, positions):
    """cache [blocks, Hkv, 16, hd] at a sequence's positions -> [n, Hkv, hd]."""
    positions = np.asarray(positions)
    return np.asarray(cache)[np.asarray(table_row)[positions // PAGE], :, positions % PAGE].astype(np.float64)


def window_attn(q, k_cache, v_cache, table, starts, lens, prefix, window: int, sinks: int, scale: float):
    """q [T, Hq, hd]; sequence b's lens[b] tokens from row starts[b] stand at positions prefix[b] ...  Returns
    o [T, Hq, hd] (zero where no sequence has a token), and what bounds its error: per row and column the mean of |v|
    under the same weights, and per row the largest sum of |scale q k|."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, hd = q.shape
    group = Hq // np.asarray(k_cache).shape[1]
    o, size, reach = np.zeros((T, Hq, hd)), np.zeros((T, Hq, hd)), np.zeros((T, Hq, 1))
    for b, (start, n, P) in enumerate(zip(starts, lens, prefix)):
        for i in range(int(n)):
            at = visible(int(P) + i, window, sinks)
            k, v = rows(k_cache, table[b], at), rows(v_cache, table[b], at)
            for h in range(Hq):
                x = q[start + i, h]
                s = scale * (k[:, h // group] @ x)
                w = np.exp(s - s.max())
                w /= w.sum()
                o[start + i, h] = w @ v[:, h // group]
                size[start + i, h] = w @ np.abs(v[:, h // group])
                reach[start + i, h, 0] = (abs(scale) * (np.abs(k[:, h // group]) @ np.abs(x))).max()
    return o, size, reach


def accept_sample(parents, tokens, target, draft, uniforms, Lmax: int):
    """One tree: (accepted path, next token), or None where the last row has no positive entry."""
    target = np.fmax(np.asarray(target, dtype=np.float64), 0.0)
    draft = None if draft is None else np.fmax(np.asarray(draft, dtype=np.float64), 0.0)
    u = np.asarray(uniforms, dtype=np.float64)
    N, V = target.shape
    path = [0]
    while True:
        node = path[-1]
        p = target[node]
        R, M, went = p.copy(), 1.0, None
        if len(path) < Lmax:
            for c in range(node + 1, N):
                if parents[c] != node:
                    continue
                x = int(tokens[c])
                known = 0 <= x < V
                q = 1.0 if draft is None else draft[node, x] if known else 0.0
                if known and u[c] * q * M < R[x]:
                    went = c
                    break
                if draft is not None:
                    R = np.maximum(R - M * draft[node], 0.0)
                    M = R.sum()
                    if not M > 0:
                        R, M = p.copy(), 1.0
                elif known:
                    M -= R[x]
                    R[x] = 0.0
        if went is None:
            break
        path.append(went)
    if not R.sum() > 0:
        R = p
    sums = np.cumsum(R)
    if not sums[-1] > 0:
        return None
    past = np.nonzero(sums > u[0] * sums[-1])[0]
    return path, int(past[0]) if past.size else int(np.nonzero(R > 0)[0][-1])
