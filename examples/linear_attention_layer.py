"""One layer of linear attention with a decay, served: a batch of prompts, then token by token.

    python examples/linear_attention_layer.py [--tokens 8]

The layer is the mixer of a hybrid model around its projections (plain matrix products here, with
random weights):

    x = rmsnorm(r) w_in                                    the norm before the block
    q, k, v, z, a = x W_in                                 one projection; its slices go to the calls as they lie
    o, S = linear attention(q, k, v, alpha(a), S)          tv_linear_attn_prompt / tv_linear_attn_step
    y = (rmsnorm(o) w_head * silu(z)) W_out                tv_gated_rmsnorm
    r = r + y,  x' = rmsnorm(r) w_next                     tv_residual_rmsnorm

After the prompts the state of every sequence is its row of S, and a new token costs one pass over it.
The single-token calls are captured into a CUDA graph and replayed.  At the end the sequences are run
again as whole prompts; their last outputs agree with the ones that came token by token.
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

EPS = 1e-6


class Layer:
    def __init__(self, width: int, heads: int, key_heads: int, dk: int, dv: int, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, scale):
            return (scale * torch.randn(*shape, generator=g, device=device)).bfloat16()

        self.H, self.Hk, self.dk, self.dv = heads, key_heads, dk, dv
        # the projection's rows are whole multiples of 16 bytes, as the calls on its slices want them
        self.split = [key_heads * dk, key_heads * dk, heads * dv, heads * dv, heads, -heads % 8]
        self.w_in = weight(width, sum(self.split), scale=width ** -0.5)
        self.w_out = weight(heads * dv, width, scale=(heads * dv) ** -0.5)
        self.n_head, self.n_next = (1 + weight(d, scale=0.1) for d in (dv, width))

    def project(self, x):
        q, k, v, z, a, _ = (x @ self.w_in).split(self.split, dim=1)
        q, k = q.unflatten(1, (self.Hk, self.dk)), k.unflatten(1, (self.Hk, self.dk))
        v, z = v.unflatten(1, (self.H, self.dv)), z.unflatten(1, (self.H, self.dv))
        return q, k, v, z, torch.sigmoid(a.float() + 3)

    def finish(self, o, z, residual):
        y = torch.empty_like(o)
        tv.tv_gated_rmsnorm(o, z, self.n_head, y, EPS)
        out, x = torch.empty_like(residual), torch.empty(residual.shape, dtype=torch.bfloat16, device=o.device)
        tv.tv_residual_rmsnorm(y.flatten(1) @ self.w_out, residual, out, EPS, out=x, weight=self.n_next)
        return out, x

    def prompts(self, x, residual, cu_seqlens, longest: int, S):
        """x, residual [T, width] of packed prompts; S [B, H, dv, dk] receives their states."""
        q, k, v, z, alpha = self.project(x)
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        err = torch.empty(S.shape[0], dtype=torch.int32, device=v.device)
        tv.tv_linear_attn_prompt(q, k, v, alpha, cu_seqlens, o, S, err, max_len=longest, q_scale=self.dk ** -0.5)
        return self.finish(o, z, residual), err

    def token(self, x, residual, S):
        """x, residual [B, width]: the next token of every sequence; S is updated in place."""
        q, k, v, z, alpha = self.project(x)
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        tv.tv_linear_attn_step(q, k, v, alpha, S, o, q_scale=self.dk ** -0.5)
        return self.finish(o, z, residual)


def serve(lengths=(300, 1, 77, 129), tokens: int = 8, width: int = 512, heads: int = 8, key_heads: int = 4, dk: int = 128,
          dv: int = 128):
    """Runs the layer and returns the largest difference between the token-by-token outputs and the
    whole prompts', relative to their root mean square."""
    dev, B = "cuda", len(lengths)
    layer = Layer(width, heads, key_heads, dk, dv)
    g = torch.Generator(device=dev).manual_seed(1)
    rows = [torch.randn(n + tokens, width, generator=g, device=dev).bfloat16() for n in lengths]

    def packed(pieces):
        ends = torch.tensor([0] + [len(p) for p in pieces]).cumsum(0).to(device=dev, dtype=torch.int32)
        return torch.cat(pieces), ends, max(len(p) for p in pieces)

    S = torch.empty(B, heads, dv, dk, device=dev)
    x, ends, longest = packed([r[:n] for r, n in zip(rows, lengths)])
    _, err = layer.prompts(x, x.float(), ends, longest, S)

    # one token of every sequence, captured once and replayed with new inputs
    x_in, r_in = torch.zeros(B, width, device=dev, dtype=torch.bfloat16), torch.zeros(B, width, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.token(x_in, r_in, S.clone())  # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r_out, x_out = layer.token(x_in, r_in, S)
    got = []
    for t in range(tokens):
        x_in.copy_(torch.stack([r[n + t] for r, n in zip(rows, lengths)]))
        r_in.copy_(x_in.float())
        graph.replay()
        got.append(torch.cat([r_out, x_out.float()], 1))

    whole = torch.empty_like(S)
    x, ends, longest = packed(rows)
    (r_all, x_all), err2 = layer.prompts(x, x.float(), ends, longest, whole)
    torch.cuda.synchronize()
    if err.any() or err2.any():
        raise RuntimeError(f"prompt errors {err.tolist()} {err2.tolist()}")
    both = torch.cat([r_all, x_all.float()], 1)
    worst = 0.0
    for t in range(tokens):
        want = both[ends[1:].long() - tokens + t]
        worst = max(worst, float((got[t] - want).abs().max() / want.square().mean().sqrt()))
    return worst, float((S - whole).norm() / whole.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8)
    outputs, states = serve(tokens=ap.parse_args().tokens)
    print(f"token by token against whole prompts: outputs differ by at most {outputs:.2e} of their rms, states by {states:.2e}")
