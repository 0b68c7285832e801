"""Acceptance by probabilities where a sum meets its border: rows whose second half repeats the first, drawn from at
one half.  Every CTA of a sequence's cluster has to decide alike, or the token is written by none of them, or by two.

Sums are carried to 2^-44 of their total, so a token is right if its share of the row, from the sum in front of it to the sum
with it, comes within that of half the total; the token does not change from call to call."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNWRITTEN = -12345


def draw(target, draft, tokens, u):
    """One call on trees of one node, or of a node and a child; err, length, next token."""
    B, N, V = target.shape
    parents = torch.tensor([[-1, 0][:N]] * B, dtype=torch.int32, device=DEV)
    out = [torch.full(s, UNWRITTEN, dtype=torch.int32, device=DEV) for s in ((B, N), (B,), (B,), (B,))]
    tv.tv_accept_sample(parents, tokens, target, draft, u, *out)
    torch.cuda.synchronize()
    return out[3].tolist(), out[1].tolist(), out[2].cpu().numpy()


def halves(B, V, mirrored, seed):
    g = torch.Generator().manual_seed(seed)
    r = torch.softmax(5.0 * torch.randn(B, V // 2, generator=g), -1)
    return torch.cat([r, r.flip(-1) if mirrored else r], -1)


def at_the_border(R, u, token):
    R = R.astype(np.float64)
    sums = np.cumsum(R)
    want, near = u * sums[-1], 2.0 ** -44 * sums[-1]
    return R[token] > 0 and sums[token] > want - near and sums[token] - R[token] < want + near


# clusters of eight CTAs for two and eight sequences, of four for 40 and 60, of two for 150
@pytest.mark.parametrize("B,V", [(2, 131072), (8, 131072), (40, 32768), (60, 16384), (150, 8192)])
@pytest.mark.parametrize("mirrored", [False, True])
def test_draws_from_halves_that_are_alike(B, V, mirrored):
    for seed in range(6):
        p = halves(B, V, mirrored, seed)
        target, tokens = p[:, None].contiguous().to(DEV), torch.zeros(B, 1, dtype=torch.int32, device=DEV)
        u = torch.full((B, 1), 0.5, device=DEV)
        err, length, first = draw(target, None, tokens, u)
        assert err == [0] * B and length == [1] * B
        for b in range(B):
            assert first[b] != UNWRITTEN and at_the_border(p[b].numpy(), 0.5, first[b]), b
        for _ in range(5):
            assert np.array_equal(draw(target, None, tokens, u)[2], first)


@pytest.mark.parametrize("mirrored", [False, True])
def test_draws_from_what_a_refusal_left(mirrored):
    # p and q each of two halves alike, so that p - q is too; the child has no probability and is refused
    B, V = 8, 131072
    for seed in range(6):
        p, q = halves(B, V, mirrored, seed), halves(B, V, mirrored, 100 + seed)
        p[:, 0] = p[:, V - 1 if mirrored else V // 2] = 0.0
        target, draft = (x[:, None].expand(B, 2, V).contiguous().to(DEV) for x in (p, q))
        tokens, u = torch.zeros(B, 2, dtype=torch.int32, device=DEV), torch.full((B, 2), 0.5, device=DEV)
        err, length, first = draw(target, draft, tokens, u)
        assert err == [0] * B and length == [1] * B
        R = np.maximum(p.numpy().astype(np.float64) - q.numpy().astype(np.float64), 0.0)
        for b in range(B):
            assert first[b] != UNWRITTEN and at_the_border(R[b], 0.5, first[b]), b
        for _ in range(5):
            assert np.array_equal(draw(target, draft, tokens, u)[2], first)
