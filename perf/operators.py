"""Measured cases of the linear-attention mixer's operators, with their plain forms.

The operators are what a layer of linear attention with a decay needs around its projections:

* ``prompt``: whole prompts, packed back to back: S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = S_t q_t;
* ``step``: the same recurrence for one new token of each sequence, the state updated in place;
* ``gated_norm``: the mixer's output normalised per head and multiplied by its gate;
* ``residual_norm``: a block's output, normalised, gated and scaled into the residual stream, with
  the next block's norm.

Heads of 64 or 128 columns, 16 heads and batches of 64 are this repository's own sizes; widths of
the residual stream are generic.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CHUNK = 128  # tokens per chunk of the plain form


def listed():
    prompt = dict(op="prompt", dk=128, dv=128, io="bf16", state="bf16", decay="token", fused=True, fresh=True)
    step = dict(op="step", dk=128, dv=128, io="bf16", state="bf16", decay="token", idle=False)
    return [
        # one short chat turn on a small layer: latency
        dict(prompt, name="prompt short", B=1, longest=200, ragged=False, Hk=16, H=16),
        # a batch of prompts as they arrive, one of them empty, continuing kept fp32 states;
        # two value heads read one key head
        dict(prompt, name="prompt ragged", B=8, longest=3001, ragged=True, Hk=16, H=32, state="f32", fresh=False),
        # one long document, one fixed decay for each head
        dict(prompt, name="prompt long", B=1, longest=32768, ragged=False, Hk=32, H=32, decay="head"),
        # a full batch of equal prompts
        dict(prompt, name="prompt batch", B=32, longest=2048, ragged=False, Hk=32, H=32),
        # fp32 throughout, narrow keys, an odd length
        dict(prompt, name="prompt fp32", B=4, longest=777, ragged=True, Hk=8, H=8, dk=64, io="f32", state="f32",
             fused=False, fresh=False),
        # one sequence decodes: latency
        dict(step, name="step single", B=1, Hk=16, H=16),
        # the batch of the repository's benchmark
        dict(step, name="step batch", B=64, Hk=16, H=32),
        # a padded batch of fp32 states, some of whose rows hold no sequence
        dict(step, name="step padded", B=200, Hk=16, H=16, state="f32", idle=True),
        # the mixer's output norm behind a decode step, and behind a batch of prompts
        dict(op="gated_norm", name="gated norm decode", rows=64, H=32, d=128, io="bf16", gate_first=False),
        dict(op="gated_norm", name="gated norm prompt", rows=40001, H=32, d=128, io="bf16", gate_first=False),
        # between two blocks behind a decode step; and behind a batch of prompts, with an fp32 residual stream
        dict(op="residual_norm", name="residual norm decode", rows=64, D=4096, io="bf16", residual="bf16", post=False,
             gate=False),
        dict(op="residual_norm", name="residual norm prompt", rows=30011, D=5120, io="bf16", residual="f32", post=True,
             gate=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "step", "gated_norm", "residual_norm"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("prompt", "step"):
        H = rng.choice([4, 6, 8, 16, 24, 32])
        c = dict(op=op, Hk=H // rng.choice([1, 1, 2]), H=H, dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]),
                 io=io, state=rng.choice(["bf16", "f32"]) if io == "bf16" else "f32", decay=rng.choice(["token", "head"]))
        if op == "prompt":
            B = _spread(rng, 1, 64)
            most = min(32768, (65536 if io == "bf16" else 32768) // B)
            return dict(c, B=B, longest=_spread(rng, 1, most), ragged=rng.random() < 0.5, fused=rng.random() < 0.5,
                        fresh=rng.random() < 0.5)
        return dict(c, B=_spread(rng, 1, 256), idle=rng.random() < 0.3)
    if op == "gated_norm":
        H, d = rng.choice([1, 4, 16, 32]), rng.choice([64, 96, 128, 130, 256])
        most = (160_000_000 if io == "bf16" else 80_000_000) // (H * d)
        return dict(op=op, rows=_spread(rng, 1, min(40000, most)), H=H, d=d, io=io, gate_first=rng.random() < 0.3)
    return dict(op=op, rows=_spread(rng, 1, 30000 if io == "bf16" else 15000), D=_spread(rng, 256, 5120), io=io,
                residual=rng.choice(["bf16", "f32"]) if io == "bf16" else "f32", post=rng.random() < 0.5,
                gate=rng.random() < 0.5)


def _lengths(case):
    """The prompts' lengths: the longest first; ragged ones spread over their logarithm, one of them empty."""
    if not case["ragged"]:
        return [case["longest"]] * case["B"]
    rng = random.Random(1000 * case["B"] + case["longest"])
    lens = [case["longest"]] + [_spread(rng, 1, case["longest"]) for _ in range(case["B"] - 1)]
    if case["B"] >= 4:
        lens[case["B"] // 2] = 0
    return lens


def work(case):
    size = {"bf16": 2, "f32": 4}
    io = size[case["io"]]
    if case["op"] in ("prompt", "step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        states = case["B"] * H * dk * dv * size[case["state"]]
        tokens = sum(_lengths(case)) if case["op"] == "prompt" else case["B"]
        live = tokens
        if case["op"] == "step" and case["idle"]:
            live = sum(_live(case))
            states = states * live // case["B"]
        alpha = 4 * H * (live if case["decay"] == "token" else 1)
        passes = 2 if case["op"] == "step" or not case["fresh"] else 1
        return {"bytes": live * (2 * Hk * dk + 2 * H * dv) * io + alpha + passes * states, "flops": 4 * live * H * dk * dv}
    if case["op"] == "gated_norm":
        n = case["rows"] * case["H"] * case["d"]
        return {"bytes": 3 * n * io + case["d"] * io, "flops": 12 * n}
    n = case["rows"] * case["D"]
    moved = io * (2 + case["gate"]) + 2 * size[case["residual"]]
    return {"bytes": n * moved + case["D"] * io * (1 + case["post"]), "flops": 12 * n}


def _live(case):
    """Which rows of a padded step hold a sequence: about four of five, the first always."""
    rng = random.Random(case["B"])
    return [True] + [rng.random() < 0.8 for _ in range(case["B"] - 1)]


def _inputs(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    io = TYPES[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    if case["op"] == "gated_norm":
        R, H, d = case["rows"], case["H"], case["d"]
        # the gate is a slice of the layer's fused projection
        proj = normal(R, H * d + 64).to(io)
        return dict(x=(normal(R, H, d) * 0.3).to(io), gate=proj[:, 64:].unflatten(1, (H, d)),
                    weight=(1 + 0.1 * normal(d)).to(io), out=torch.zeros(R, H, d, device=DEVICE, dtype=io))
    if case["op"] == "residual_norm":
        R, D = case["rows"], case["D"]
        res = TYPES[case["residual"]]
        return dict(y=normal(R, D).to(io), residual=(3 * normal(R, D)).to(res),
                    post=(1 + 0.1 * normal(D)).to(io) if case["post"] else None,
                    gate=torch.sigmoid(normal(R, D)).to(io) if case["gate"] else None,
                    weight=(1 + 0.1 * normal(D)).to(io), scale=0.7,
                    residual_out=torch.zeros(R, D, device=DEVICE, dtype=res), out=torch.zeros(R, D, device=DEVICE, dtype=io))

    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    state = TYPES[case["state"]]
    lens = _lengths(case) if case["op"] == "prompt" else [1] * B
    T = sum(lens)
    unit = torch.nn.functional.normalize
    q, k, v = (unit(normal(T, Hk, dk), dim=-1).to(io), unit(normal(T, Hk, dk), dim=-1).to(io), normal(T, H, dv).to(io))
    if case.get("fused"):  # slices of one projection's output
        whole = torch.cat([x.flatten(1) for x in (q, k, v)], dim=1)
        q, k, v = whole.split([Hk * dk, Hk * dk, H * dv], dim=1)
        q, k, v = q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (H, dv))
    # heads forget over spans from a token or two to thousands of tokens
    span = 2.0 ** -torch.linspace(0, 11, H, device=DEVICE)
    alpha = 1 - span / 2 if case["decay"] == "head" else torch.exp(-torch.nn.functional.softplus(normal(T, H)) * span)
    S = (0.02 * normal(B, H, dv, dk)).to(state)
    st = dict(q=q, k=k, v=v, alpha=alpha, out=torch.zeros(T, H, dv, device=DEVICE, dtype=io),
              err=torch.zeros(B, device=DEVICE, dtype=torch.int32), q_scale=dk ** -0.5)
    if case["op"] == "step":
        st["S"] = S
        st["live"] = torch.tensor(_live(case), device=DEVICE, dtype=torch.int32) if case["idle"] else None
        return st
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    st.update(S0=None if case["fresh"] else S, S=torch.zeros_like(S), longest=max(lens),
              cu_seqlens=torch.tensor(ends, device=DEVICE, dtype=torch.int32))
    return st


def prepare(case, seed):
    return dict(_inputs(case, seed), op=case["op"], gate_first=case.get("gate_first", False))


def run(st):
    return {"prompt": _prompt, "step": _step, "gated_norm": _gated_norm, "residual_norm": _residual_norm}[st["op"]](st)


def _prompt(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_linear_attn_prompt(st["q"], st["k"], st["v"], st["alpha"], st["cu_seqlens"], st["out"], st["S"], st["err"],
                                 S0=st["S0"], max_len=st["longest"], q_scale=st["q_scale"])
        return {"out": st["out"], "S": st["S"]}
    # Chunked: within a chunk the masked, decayed scores; across chunks the states at the chunks' starts.
    v, cu = st["v"].float(), st["cu_seqlens"].long()
    T, H, dv = v.shape
    heads = torch.arange(H, device=v.device) // (H // st["q"].shape[1])
    q, k = st["q"].float()[:, heads] * st["q_scale"], st["k"].float()[:, heads]
    B, chunks = cu.numel() - 1, max(1, -(-st["longest"] // CHUNK))
    at = torch.arange(chunks * CHUNK, device=v.device)
    valid = at < (cu[1:] - cu[:-1])[:, None]
    place = torch.where(valid, cu[:-1, None] + at, 0)

    def cut(x):  # [T, H, ...] -> [B, H, chunks, CHUNK, ...], zero past a prompt's end
        x = x[place] * valid.reshape(B, -1, *[1] * (x.dim() - 1)).to(x.dtype)
        return x.unflatten(1, (chunks, CHUNK)).movedim(3, 1)

    qc, kc, vc = cut(q), cut(k), cut(v)
    log = cut(torch.log(st["alpha"].double()).expand(T, H))
    g = torch.cumsum(log, -1)  # log of the decay from before the chunk to each token
    gap = g[..., :, None] - g[..., None, :]
    seen = torch.ones(CHUNK, CHUNK, device=v.device, dtype=torch.bool).tril()
    scores = (qc @ kc.transpose(-1, -2)) * torch.exp(torch.where(seen, gap, -math.inf)).float()
    grown = (vc * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(-1, -2) @ kc
    total = torch.cumsum(g[..., -1], -1)
    before = torch.cat([torch.zeros_like(total[..., :1]), total], -1)  # to the start of chunk c = 0 .. chunks
    order = torch.arange(chunks + 1, device=v.device)
    gap = before[..., :, None] - total[..., None, :]
    carry = torch.exp(torch.where(order[:, None] > order[:-1], gap, -math.inf)).float()
    starts = (carry @ grown.flatten(-2)).unflatten(-1, grown.shape[-2:])
    if st["S0"] is not None:
        starts = starts + torch.exp(before).float()[..., None, None] * st["S0"].float()[:, :, None]
    o = scores @ vc + torch.exp(g).float()[..., None] * (qc @ starts[:, :, :-1].transpose(-1, -2))
    o = o.flatten(2, 3).transpose(1, 2)  # [B, tokens, H, dv]
    token = torch.arange(T, device=v.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    return {"out": o[seq, token - cu[seq]].to(st["out"].dtype), "S": starts[:, :, -1].to(st["S"].dtype)}


def _step(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_linear_attn_step(st["q"], st["k"], st["v"], st["alpha"], st["S"], st["out"], live=st["live"],
                               q_scale=st["q_scale"])
        return {"out": st["out"], "S": st["S"]}
    v, S = st["v"].float(), st["S"].float()
    B, H, _ = v.shape
    heads = torch.arange(H, device=v.device) // (H // st["q"].shape[1])
    q, k = st["q"].float()[:, heads] * st["q_scale"], st["k"].float()[:, heads]
    new = st["alpha"].expand(B, H)[..., None, None] * S + v[..., :, None] * k[..., None, :]
    o = (new * q[..., None, :]).sum(-1).to(st["out"].dtype)
    new = new.to(st["S"].dtype)
    if st["live"] is not None:
        live = st["live"].bool()[:, None, None]
        o, new = torch.where(live, o, st["out"]), torch.where(live[..., None], new, st["S"])
    st["S"].copy_(new)
    return {"out": o, "S": st["S"]}


def _gated_norm(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_gated_rmsnorm(st["x"], st["gate"], st["weight"], st["out"], EPS, gate_first=st["gate_first"])
        return st["out"]
    x, gate, w = st["x"].float(), st["gate"].float(), st["weight"].float()
    gate = gate / (1 + torch.exp(-gate))
    x = x * gate if st["gate_first"] else x
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return (x if st["gate_first"] else x * gate).to(st["out"].dtype)


def _residual_norm(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_residual_rmsnorm(st["y"], st["residual"], st["residual_out"], EPS, out=st["out"], weight=st["weight"],
                               post_weight=st["post"], gate=st["gate"], scale=st["scale"])
        return {"residual": st["residual_out"], "out": st["out"]}
    y = st["y"].float()
    if st["post"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * st["post"].float()
    if st["gate"] is not None:
        y = y * st["gate"].float()
    r = st["residual"].float() + st["scale"] * y
    out = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * st["weight"].float()
    return {"residual": r.to(st["residual_out"].dtype), "out": out.to(st["out"].dtype)}


def exact(case, seed):
    """The definitions in 64 bits: the recurrences token by token."""
    st = _inputs(case, seed)
    if case["op"] == "gated_norm":
        x, gate, w = (st[n].double() for n in ("x", "gate", "weight"))
        act = gate * torch.sigmoid(gate)
        x = x * act if case["gate_first"] else x
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        return n if case["gate_first"] else n * act
    if case["op"] == "residual_norm":
        y, r = st["y"].double(), st["residual"].double()
        if case["post"]:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * st["post"].double()
        r = r + st["scale"] * (y * st["gate"].double() if case["gate"] else y)
        return {"residual": r, "out": r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * st["weight"].double()}
    B, H, group = case["B"], case["H"], case["H"] // case["Hk"]
    T = st["v"].shape[0]
    q, k = (st[n].double().repeat_interleave(group, dim=1) for n in ("q", "k"))
    v, alpha = st["v"].double(), st["alpha"].double().expand(T, H)
    out = torch.zeros(T, H, case["dv"], device=DEVICE, dtype=torch.float64)
    start = st["S"] if case["op"] == "step" else st["S0"]
    S = torch.zeros(B, H, case["dv"], case["dk"], device=DEVICE, dtype=torch.float64) if start is None else start.double()
    lens = _lengths(case) if case["op"] == "prompt" else [int(x) for x in _live(case)] if case["idle"] else [1] * B
    first = [sum(lens[:b]) for b in range(B)] if case["op"] == "prompt" else list(range(B))
    # longest sequences first: at token t the first n of them are still running
    order = sorted(range(B), key=lambda b: -lens[b])
    at = torch.tensor([first[b] for b in order], device=DEVICE)
    S = S[order].clone()
    n = B
    for t in range(max(lens)):
        while n and lens[order[n - 1]] <= t:
            n -= 1
        i = at[:n] + t
        S[:n].mul_(alpha[i][..., None, None]).addcmul_(v[i][..., :, None], k[i][..., None, :])
        out[i] = (S[:n] @ q[i][..., None])[..., 0]
    back = sorted(range(B), key=lambda j: order[j])
    return {"out": out * st["q_scale"], "S": S[back]}
