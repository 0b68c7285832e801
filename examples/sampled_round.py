"""Sampled speculative rounds over softmax attention with a window: a draft model proposes, the target verifies.

    python examples/sampled_round.py [--rounds 6]

Both models are one attention layer between a table of token vectors and a head (random weights):

    q, k, v = E[token] W_in
    q, k = rotated rmsnorm(q), rmsnorm(k); k and v into the paged cache      tv_qk_norm_rope
    o = attention over the cache, a window and a few first tokens            tv_window_attn_prompt / tv_window_attn_step
    p = softmax((E[token] + o W_out) W_head)

A round: the draft model takes its last token and draws k more, one at a time (tv_accept_sample with a single node draws
one token); the target takes the last token and the k drafted ones as one chain behind its cache; tv_accept_sample keeps
what stands and draws the token after it.  Refused tokens need no undoing: their slots are written again by the next round.
At the end the committed tokens are run through the target as whole prompts, and their outputs agree with the rounds'.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import tree_speculative_verification_gdn_gb300 as tv  # noqa: E402

EPS, THETA = 1e-6, 1e4
DEV = "cuda"


def whole(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """One layer and its paged cache with room for ``room`` tokens of each of B sequences."""

    def __init__(self, vocab, width, Hq, Hkv, hd, B, room, window, sinks, seed, like=None, noise=0.3):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def weight(*shape, scale):
            return scale * torch.randn(*shape, generator=g, device=DEV)

        self.Hq, self.Hkv, self.hd, self.window, self.sinks = Hq, Hkv, hd, window, sinks
        self.table_in = weight(vocab, width, scale=1.0)
        self.head = weight(width, vocab, scale=2 * width ** -0.5)
        self.w_in = weight(width, (Hq + 2 * Hkv) * hd, scale=width ** -0.5)
        self.w_out = weight(Hq * hd, width, scale=(Hq * hd) ** -0.5)
        if like is not None:  # a draft has its target's opinion, more or less
            for n in ("table_in", "head", "w_in", "w_out"):
                setattr(self, n, getattr(like, n) + noise * getattr(self, n))
        self.norms = [(1 + weight(hd, scale=0.1)).bfloat16() for _ in range(2)]
        blocks = -(-room // 16)
        self.k_cache, self.v_cache = (torch.zeros(B * blocks, Hkv, 16, hd, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        self.block_table = torch.randperm(B * blocks, generator=g, device=DEV).to(torch.int32).view(B, blocks)

    def rotated(self, x, prefix, cu):
        Hq, Hkv, hd = self.Hq, self.Hkv, self.hd
        q, k, v = (x @ self.w_in).bfloat16().split([Hq * hd, Hkv * hd, Hkv * hd], dim=1)
        out = torch.empty(len(x), Hq, hd, device=DEV, dtype=torch.bfloat16)
        err = torch.empty_like(prefix)
        tv.tv_qk_norm_rope(q.unflatten(1, (Hq, hd)), k.unflatten(1, (Hkv, hd)), out, prefix, err, v=v.unflatten(1, (Hkv, hd)),
                           k_cache=self.k_cache, v_cache=self.v_cache, block_table=self.block_table, cu_seqlens=cu,
                           q_weight=self.norms[0], k_weight=self.norms[1], eps=EPS, rope_theta=THETA)
        return out, err

    def probs(self, x, o):
        return torch.softmax((x + o.float().flatten(1) @ self.w_out) @ self.head, dim=-1)

    def chains(self, tokens, cu, prefix, longest):
        """tokens [T] packed by cu behind prefix [B] cached ones: probabilities [T, vocab], attention outputs, errors."""
        x = self.table_in[tokens.long()]
        q, err = self.rotated(x, prefix, cu)
        o, err2 = torch.empty_like(q), torch.empty_like(err)
        tv.tv_window_attn_prompt(q, self.k_cache, self.v_cache, self.block_table, cu, prefix, o, err2, window=self.window,
                                 sinks=self.sinks, max_len=longest)
        return self.probs(x, o), o, err + err2

    def one(self, tokens, prefix):
        """One token of each sequence."""
        x = self.table_in[tokens.long()]
        q, err = self.rotated(x, prefix, None)
        o, err2 = torch.empty_like(q), torch.empty_like(err)
        tv.tv_window_attn_step(q, self.k_cache, self.v_cache, self.block_table, prefix, o, err2, window=self.window,
                               sinks=self.sinks)
        return self.probs(x, o), err + err2


def accept(parents, tokens, target, draft, uniforms):
    B, N = parents.shape
    path, length, after, err = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((B, N), (B,), (B,), (B,)))
    tv.tv_accept_sample(parents, tokens, target, draft, uniforms, path, length, after, err)
    return path, length, after, err


def serve(lengths=(40, 1, 133), rounds: int = 6, drafts: int = 4, vocab: int = 500, width: int = 256, Hq: int = 4, Hkv: int = 2,
          hd: int = 64, window: int = 50, sinks: int = 3, seed: int = 0, watch=None):
    """Runs prompts and rounds; returns the committed tokens of each sequence and how far the rounds' attention outputs are
    from those of the whole sequences run as prompts, relative to their norm.  ``watch`` is called with every acceptance's
    inputs and outputs."""
    B, room = len(lengths), max(lengths) + (rounds + 1) * (drafts + 1)
    target = Model(vocab, width, Hq, Hkv, hd, B, room, window, sinks, seed)
    draft = Model(vocab, width, Hq, Hkv, hd, B, room, window, sinks, seed + 1, like=target)
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    said = [torch.randint(vocab, (n,), generator=g, device=DEV).tolist() for n in lengths]
    prefix, errors = whole([0] * B), []

    # the prompts, and the first token behind them
    cu = whole([0] + lengths_to(lengths))
    tokens = whole([t for s in said for t in s])
    p, o, err = target.chains(tokens, cu, prefix, max(lengths))
    errors += [err, draft.chains(tokens, cu, prefix, max(lengths))[2]]
    seen = [[o[a:b]] for a, b in zip(cu[:-1].tolist(), cu[1:].tolist())]
    rows = p[(cu[1:] - 1).long()]
    last = accept(whole([[-1]] * B), whole([[0]] * B), rows[:, None].contiguous(), None, torch.rand(B, 1, generator=g, device=DEV))[2]
    prefix = whole(lengths)
    chain = whole([list(range(-1, drafts))] * B)
    ends = whole([i * (drafts + 1) for i in range(B + 1)])
    for _ in range(rounds):
        # the draft's tokens, each drawn from its probabilities behind the one before
        proposed, opinion = [last], []
        for i in range(drafts + 1):  # once more, so that the last drafted token too lies in the draft's cache
            p, err = draft.one(proposed[-1], prefix + i)
            errors.append(err)
            opinion.append(p)
            if i < drafts:
                proposed.append(accept(whole([[-1]] * B), whole([[0]] * B), p[:, None].contiguous(), None,
                                       torch.rand(B, 1, generator=g, device=DEV))[2])
        tokens, q = torch.stack(proposed, 1).contiguous(), torch.stack(opinion, 1).contiguous()
        p, o, err = target.chains(tokens.flatten(), ends, prefix, drafts + 1)
        p = p.view(B, drafts + 1, vocab)
        u = torch.rand(B, drafts + 1, generator=g, device=DEV)
        path, length, after, err2 = accept(chain, tokens, p, q, u)
        errors += [err, err2]
        if watch is not None:
            watch(chain, tokens, p, q, u, path, length, after)
        for b, n in enumerate(length.tolist()):
            said[b] += tokens[b, :n].tolist()
            seen[b].append(o.view(B, drafts + 1, Hq, hd)[b, :n])
        prefix, last = prefix + length, after
    # the committed tokens as whole prompts in a cache of their own
    fresh = Model(vocab, width, Hq, Hkv, hd, B, room, window, sinks, seed)
    counts = [len(s) for s in said]
    _, o, err = fresh.chains(whole([t for s in said for t in s]), whole([0] + lengths_to(counts)), whole([0] * B), max(counts))
    errors.append(err)
    if torch.cat(errors).any():
        raise RuntimeError("a call reported an error")
    got = torch.cat([torch.cat(s) for s in seen]).double()
    return said, float((got - o.double()).norm() / o.double().norm())


def lengths_to(lengths):
    ends = []
    for n in lengths:
        ends.append((ends[-1] if ends else 0) + n)
    return ends


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=6)
    args = ap.parse_args()
    tokens, off = serve(rounds=args.rounds)
    print(f"{[len(t) for t in tokens]} tokens after {args.rounds} rounds; the rounds' outputs are off the whole prompts' by {off:.2e}")
