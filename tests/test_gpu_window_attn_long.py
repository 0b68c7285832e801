"""Windowed attention over long contexts: a few pages of keys stand at millions of positions, so that the 64-bit result is a
sum over distinct keys, each as often as it is seen.  Values lie around 1: a sum that falls short shows.

Bounds, of A, the mean of |v| under the weights, beside those of short contexts (tests/_window.py): a matrix unit may cut up to
2^-23 of a sum with each 16 keys that it adds.  It adds 2^15 keys to a sum at most, and half of the cuts count as the sum
grows: 2^-13 in all; sums of 2^15 keys are added in fp32, some hundred of them: 2^-16."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import BF, DEV, U, f64, whole

pytestmark = pytest.mark.gpu


def make(lens, prefix, Hq, Hkv, hd, seed, growing):
    """Sequences over the same 32 blocks; ``growing``: the keys of each quarter of a context are larger than the last one's."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(32, Hkv, 16, hd, generator=g) for _ in range(2))
    if growing:
        k *= torch.tensor([0.5, 1.0, 1.5, 2.0]).repeat_interleave(8)[:, None, None, None]
    rng = np.random.default_rng(seed)
    pages = -(-(max(p + n for p, n in zip(prefix, lens))) // 16)
    table = rng.integers(0, 8, size=(len(lens), pages))
    table += (np.arange(pages) * 4 // pages * 8)[None] if growing else rng.integers(0, 4, size=table.shape) * 8
    q = torch.randn(sum(lens), Hq, hd, generator=g)
    return [x.to(BF).to(DEV) for x in (q, k, 1 + 0.25 * v)], whole(table), table


def want(q, k, v, table, lens, prefix):
    """(o, A, S): the largest sum of |scale q k| of a row, as tests/_window.py has them."""
    q, k, v = (torch.from_numpy(f64(x)).to(DEV) for x in (q, k, v))
    Hkv, hd = k.shape[1], k.shape[3]
    q = q.unflatten(1, (Hkv, -1))
    k, v = (x.transpose(0, 1).flatten(1, 2) for x in (k, v))                      # [Hkv, keys, hd]
    o, size, reach, start = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q[..., :1]), 0
    for b, (n, P) in enumerate(zip(lens, prefix)):
        of = torch.from_numpy(table[b]).to(DEV).repeat_interleave(16) * 16 + torch.arange(16, device=DEV).repeat(table.shape[1])
        times = torch.bincount(of[:P], minlength=k.shape[1])[None].repeat(n, 1)
        new = torch.nn.functional.one_hot(of[P:P + n], k.shape[1]).cumsum(0)
        times = (times + new).double()[:, None, None]                              # [n, 1, 1, keys]
        x = q[start:start + n]
        s = torch.einsum("nkgd,kjd->nkgj", x, k) * hd ** -0.5
        top = s.masked_fill(times == 0, -torch.inf).amax(-1, keepdim=True)
        w = times * torch.exp(s - top)
        w /= w.sum(-1, keepdim=True)
        o[start:start + n] = torch.einsum("nkgj,kjd->nkgd", w, v)
        size[start:start + n] = torch.einsum("nkgj,kjd->nkgd", w, v.abs())
        reach[start:start + n] = (torch.einsum("nkgd,kjd->nkgj", x.abs(), k.abs()) * hd ** -0.5).amax(-1, keepdim=True)
        start += n
    return [x.flatten(1, 2).cpu().numpy() for x in (o, size, reach)]


def near(out, wants, more):
    o, size, reach = wants
    hd = o.shape[-1]
    got = f64(out)
    tol = (2 * 2.0 ** -8 + 4 * (hd + 8) * U * reach + more) * size + 2.0 ** -8 * np.abs(o)
    assert np.isfinite(got).all()
    over = np.abs(got - o) - tol
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} past the bound, worst by {over.max():.3e}"
    return float(((got - o) / size).mean())


LONG = 2.0 ** -13 + 2.0 ** -16


@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("lens,prefix,Hq,Hkv", [
    ([70], [(1 << 22) + 5], 8, 2),            # units cut among the CTAs, some thousand tiles each
    ([2500], [40000], 16, 1),                 # whole units, just past one part
    ([33, 0, 1, 300], [90000, 7, 1 << 21, 32768 - 300], 6, 2),
    ([64, 64], [32768 - 64, 32769 - 64], 4, 1),
])
def test_prompts(lens, prefix, Hq, Hkv, hd, growing):
    (q, k, v), table_d, table = make(lens, prefix, Hq, Hkv, hd, hd + sum(lens), growing)
    out, err = torch.full_like(q, 7.0), torch.full((len(lens),), 9, dtype=torch.int32, device=DEV)
    tv.tv_window_attn_prompt(q, k, v, table_d, whole(np.cumsum([0] + lens)), whole(prefix), out, err)
    torch.cuda.synchronize()
    assert not err.any()
    # errors of weights and of the store go either way: their mean over thousands of outputs stays below a quarter of one
    assert abs(near(out, want(q, k, v, table, lens, prefix), LONG)) <= LONG + 2.0 ** -10
    again = torch.empty_like(out)
    tv.tv_window_attn_prompt(q, k, v, table_d, whole(np.cumsum([0] + lens)), whole(prefix), again, err)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("growing", [False, True])
# a head a CTA; some cut, some whole; one head for all CTAs
@pytest.mark.parametrize("hd,heads,before", [(64, 456, 1 << 22), (128, 304, 1 << 22), (256, 152, 1 << 22), (128, 200, 1 << 21),
                                             (256, 333, 300_000), (64, 1000, 140_000), (128, 1, 1 << 22)])
def test_single_tokens(hd, heads, before, growing):
    (q, k, v), table_d, table = make([1], [before], heads, heads, hd, hd + heads, growing)
    out, err = torch.full_like(q, 7.0), torch.full((1,), 9, dtype=torch.int32, device=DEV)
    tv.tv_window_attn_step(q, k, v, table_d, whole([before]), out, err)
    torch.cuda.synchronize()
    assert not err.any()
    assert abs(near(out, want(q, k, v, table, [1], [before]), LONG)) <= LONG + 2.0 ** -10
    again = torch.empty_like(out)
    tv.tv_window_attn_step(q, k, v, table_d, whole([before]), again, err)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
