"""Paged caches, calls and bounds of the windowed attention's GPU tests."""
import numpy as np
import torch

import tree_speculative_verification_gdn_gb300 as tv
import workloads as W
from oracle import window as O

DEV = "cuda"
U = 2.0 ** -24
BF = torch.bfloat16


def whole(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return W.f64(t.cpu())


def pages(needs, seed, spare=2, most=None):
    """(blocks, table [B, most] on the CPU): pages in any order, unused entries out of the cache."""
    needs = [-(-n // 16) for n in needs]
    blocks = sum(needs) + spare
    order = np.random.default_rng(seed).permutation(blocks)
    table = np.full((len(needs), max(1, max(needs)) if most is None else most), 1 << 30, dtype=np.int32)
    for b, n in enumerate(needs):
        table[b, :n], order = order[:n], order[n:]
    return blocks, table


def case(lens, prefix, Hq, Hkv, hd, seed=0, scale=1.5, poison=True, step=False, most=None, unseen=None):
    """Random queries and a cache that holds the keys of every position.  ``poison``: slots of no position, and the
    positions (b, first, last) in ``unseen``, hold NaN, and pages wholly in ``unseen`` have left the table."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    blocks, table = pages([p + n if n else 0 for p, n in zip(prefix, lens)], seed, most=most)
    fused = torch.randn(T, Hq * hd + 64, generator=g) * scale
    q = fused.to(BF).to(DEV)[:, 64:].unflatten(1, (Hq, hd))   # a slice of a projection's output
    caches = [torch.randn(blocks, Hkv, 16, hd, generator=g).to(BF) for _ in range(2)]
    real = table.copy()
    if poison:
        keep = torch.zeros(blocks, 16, dtype=torch.bool)
        for b, (p, n) in enumerate(zip(prefix, lens)):
            at = torch.arange(p + n if n else 0)
            for first, last in [(x, y) for s, x, y in unseen or () if s == b]:
                at = at[(at < first) | (at >= last)]
                table[b, -(-first // 16):last // 16] = -1
            keep[torch.tensor(real[b])[at // 16].long(), at % 16] = True
        for c in caches:
            c.masked_fill_(~keep[:, None, :, None], float("nan"))
    cu = np.concatenate([[0], np.cumsum(lens)])
    return dict(q=q, k=caches[0].to(DEV), v=caches[1].to(DEV), table=whole(table), real=real, cu=whole(cu), prefix=whole(prefix),
                lens=list(lens), starts=cu[:-1].tolist(), before=list(prefix), step=step, scale=hd ** -0.5)


def attend(c, window=0, sinks=0, live=None, stream=None, workspace=None, max_len=None, out=None, sm_scale=None):
    T, Hq, hd = c["q"].shape
    if out is None:
        out = torch.full((T, Hq, hd), 7.0, dtype=BF, device=DEV)
    err = torch.full((len(c["lens"]),), 9, dtype=torch.int32, device=DEV)
    if c["step"]:
        tv.tv_window_attn_step(c["q"], c["k"], c["v"], c["table"], c["prefix"], out, err, window=window, sinks=sinks,
                               live=live, stream=stream, workspace=workspace, sm_scale=sm_scale)
    else:
        tv.tv_window_attn_prompt(c["q"], c["k"], c["v"], c["table"], c["cu"], c["prefix"], out, err, window=window,
                                 sinks=sinks, max_len=max_len, stream=stream, workspace=workspace, sm_scale=sm_scale)
    torch.cuda.synchronize()
    return out, err.tolist()


def oracle(c, window, sinks, scale=None):
    k, v = (np.nan_to_num(f64(c[n])) for n in ("k", "v"))
    return O.window_attn(f64(c["q"]), k, v, c["real"], c["starts"], c["lens"], c["before"], window, sinks,
                         c["scale"] if scale is None else scale)


def check(c, out, window, sinks, rows=None, scale=None, want=None):
    """|o - oracle| <= (2 * 2^-8 + 4 (hd + 8) u S) A + 2^-8 |o|: weights and their sum in bf16 (2^-8 each), scores summed
    over hd products that the matrix units may cut instead of round (2 (hd + 8) u of S = max sum |scale q k|, twice: the
    weight and the sum of weights), the result rounded once; A the mean of |v| under the weights."""
    o, size, reach = oracle(c, window, sinks, scale) if want is None else want
    hd = o.shape[-1]
    got = f64(out)
    rows = np.arange(o.shape[0]) if rows is None else np.asarray(rows)
    tol = (2 * 2.0 ** -8 + 4 * (hd + 8) * U * reach) * size + 2.0 ** -8 * np.abs(o)
    assert np.isfinite(got[rows]).all()
    over = (np.abs(got - o) - tol)[rows]
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} past the bound, worst by {over.max():.3e}"
