"""Measured cases of a sampled verification round over windowed softmax attention, with their plain forms.

The operators are what such a round needs beside the tree calls:

* ``rotate``: norms of queries and keys per head, the rotation by position, and the new keys and values
  put into the paged cache;
* ``prompt``: attention of new tokens -- whole prompts, or drafted chains -- over that cache, within a
  window and to a few first tokens that stay visible;
* ``step``: the same for one new token of each sequence;
* ``accept``: which drafted tokens stand, by the target's and the draft's probabilities and given random
  numbers, and the token after them.

Pages of 16 tokens, 16 query heads on 4 key heads of 128 or 256 columns, batches of 32 and 64, a context of
8192 tokens and theta 1e6 are this repository's own; the other sizes are generic.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 1e6
PAGE = 16
PIECE = 1 << 31  # bytes of scores that the plain form of a prompt holds at a time
LARGEST = dict(rotate=87_000_000, prompt=550_000_000_000, step=210_000_000, accept=42_000_000)  # see _size


def listed():
    rotate = dict(op="rotate", Hq=16, Hkv=4, hd=128, rotary=128, io="bf16", cache=True, weight=True)
    prompt = dict(op="prompt", Hq=16, Hkv=4, hd=128, window=0, sinks=0, before=0)
    step = dict(op="step", Hq=16, Hkv=4, hd=128, window=0, sinks=0, idle=False)
    return [
        # behind the projections of a decode step: latency
        dict(rotate, name="rotate decode", B=64, longest=1, before=8192),
        # a batch of prompts as they arrive, into the cache
        dict(rotate, name="rotate prompts", B=8, longest=7001, before=0, Hq=32, Hkv=8),
        # a quarter of wide heads rotates, fp32, far positions, no cache behind it
        dict(rotate, name="rotate fp32", B=2, longest=1500, before=1_000_000, Hkv=2, hd=256, rotary=64, io="f32",
             cache=False, weight=False),
        # one short chat turn: latency
        dict(prompt, name="prompt short", B=1, longest=200, ragged=False),
        # prompts as they arrive, one of them empty, behind cached turns; a window and its sinks
        dict(prompt, name="prompt ragged", B=8, longest=3001, ragged=True, before=2000, window=1024, sinks=4, hd=256),
        # one long document, 32 query heads
        dict(prompt, name="prompt long", B=1, longest=16384, ragged=False, Hq=32, Hkv=8),
        # drafted chains of eight tokens behind long contexts
        dict(prompt, name="prompt chains", B=32, longest=8, ragged=False, before=8192),
        # one sequence decodes: latency
        dict(step, name="step single", B=1, before=4096),
        # the batch and context of the repository's benchmark
        dict(step, name="step batch", B=64, before=8192),
        # a padded batch with a window and sinks; pages behind the window were given back
        dict(step, name="step window", B=200, before=20000, window=2048, sinks=4, idle=True),
        # drafted chains of four tokens, the draft's probabilities known
        dict(op="accept", name="accept chain", B=64, N=5, V=131072, io="f32", shape="chain", known=True),
        # trees of the draft's most likely tokens
        dict(op="accept", name="accept tree", B=8, N=32, V=50021, io="bf16", shape="tree", known=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(case):
    """What the cost of a drawn case is bounded by: elements of queries and keys; products of prompts; elements
    of a step's keys; elements of the target's probabilities."""
    if case["op"] == "rotate":
        return sum(_lengths(case)) * (case["Hq"] + 2 * case["Hkv"]) * case["hd"] * {"bf16": 1, "f32": 2}[case["io"]]
    if case["op"] == "prompt":
        return sum(_pairs(case, p, n) for p, n in zip(_before(case), _lengths(case))) * case["Hq"] * case["hd"]
    if case["op"] == "step":
        return sum(_seen(case, p, 1) for p in _before(case)) * case["Hkv"] * case["hd"]
    return case["B"] * case["N"] * case["V"]


def draw(rng):
    while True:
        op = rng.choice(["rotate", "prompt", "prompt", "step", "step", "accept"])
        if op == "accept":
            case = dict(op=op, B=_spread(rng, 1, 64), N=_spread(rng, 1, 64), V=_spread(rng, 1000, 150_000),
                        io=rng.choice(["f32", "f32", "bf16"]), shape=rng.choice(["chain", "tree"]),
                        known=rng.random() < 0.6)
        else:
            Hkv, hd = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
            case = dict(op=op, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 4, 5, 8]), hd=hd)
            if op == "rotate":
                io = rng.choice(["bf16", "bf16", "f32"])
                case.update(B=_spread(rng, 1, 64), longest=_spread(rng, 1, 8000), before=_spread(rng, 1, 1_000_000) - 1,
                            rotary=rng.choice([hd, hd, hd // 2, hd // 4]), io=io, weight=rng.random() < 0.7,
                            cache=io == "bf16" and rng.random() < 0.7)
                if case["cache"]:
                    case["before"] = min(case["before"], 10000)
            else:
                case.update(B=_spread(rng, 1, 64 if op == "prompt" else 256), before=_spread(rng, 1, 30000) - 1,
                            window=rng.choice([0, _spread(rng, 16, 8192)]), sinks=0)
                if case["window"]:
                    case["sinks"] = rng.choice([0, 1, 4, 64, 100])
                if op == "prompt":
                    case.update(longest=_spread(rng, 1, 16384), ragged=rng.random() < 0.5)
                else:
                    case["idle"] = rng.random() < 0.3
        if _size(case) <= LARGEST[op] and (op == "accept" or _slots(case) * case["Hkv"] * case["hd"] <= 2 ** 30):
            return case


def _lengths(case):
    """New tokens of each sequence: the longest first; ragged ones spread over their logarithm, one of them empty."""
    B, longest = case["B"], case.get("longest", 1)
    if longest == 1 or not case.get("ragged", True):
        return [longest] * B
    rng = random.Random(1000 * B + longest)
    lens = [longest] + [_spread(rng, 1, longest) for _ in range(B - 1)]
    if B >= 4:
        lens[B // 2] = 0
    return lens


def _before(case):
    """Cached tokens of each sequence, from half of the case's number to all of it."""
    rng = random.Random(7 * case["B"] + case["before"])
    return [case["before"]] + [rng.randint(case["before"] // 2, case["before"]) for _ in range(case["B"] - 1)]


def _live(case):
    """Which rows of a padded batch hold a sequence: about four of five, the first always."""
    rng = random.Random(case["B"])
    return [True] + [rng.random() < 0.8 or not case["idle"] for _ in range(case["B"] - 1)]


def _first(case, p):
    """First position within the window of the query at position p."""
    return max(0, p - case["window"] + 1) if case["window"] else 0


def _seen(case, p, n):
    """Keys that the n queries from position p on see between them."""
    if n == 0:
        return 0
    lo = _first(case, p)
    return p + n - lo + min(case["sinks"], lo)


def _pairs(case, p, n):
    """Keys that each of the n queries from position p on sees, summed."""
    w, s = case["window"], case["sinks"]
    if not w:
        return n * p + n * (n + 1) // 2
    full = min(max(p + n - (w + s), 0), n)  # queries that see window and sinks whole, with keys between them hidden
    rest = n - full
    return full * (w + s) + rest * p + rest * (rest + 1) // 2


def _slots(case):
    if case["op"] == "rotate" and not case["cache"]:
        return 0
    return sum(-(-(p + n) // PAGE) * PAGE for p, n in zip(_before(case), _lengths(case)))


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "accept":
        # the row that the last token is drawn from, and what the walk looks up
        return {"bytes": case["B"] * (case["V"] * size[case["io"]] + case["N"] * 20), "flops": 2 * case["B"] * case["V"]}
    Hq, Hkv, hd, tokens = case["Hq"], case["Hkv"], case["hd"], sum(_lengths(case))
    if case["op"] == "rotate":
        n = tokens * (Hq + Hkv) * hd
        moved = n + (tokens * Hkv * hd if case["cache"] else 0)
        return {"bytes": 2 * moved * size[case["io"]], "flops": 8 * n}
    parts = [x for x, live in zip(zip(_before(case), _lengths(case)), _live(case) if case["op"] == "step" else [True] * case["B"])
             if live]
    keys, pairs = sum(_seen(case, p, n) for p, n in parts), sum(_pairs(case, p, n) for p, n in parts)
    return {"bytes": 4 * sum(n for _, n in parts) * Hq * hd + 4 * keys * Hkv * hd, "flops": 4 * pairs * Hq * hd}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _whole(values):
    return torch.tensor(values, device=DEVICE, dtype=torch.int32)


def _pages(case, seed):
    """A cache with room for every sequence, its pages in any order, and the table of them."""
    need = [-(-(p + n) // PAGE) for p, n in zip(_before(case), _lengths(case))]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.zeros(case["B"], max(max(need), 1) + 1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        del order[:n]
    return blocks, table


def _inputs(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    if case["op"] == "accept":
        return _drafts(case, g, seed)
    B, Hq, Hkv, hd = (case[n] for n in ("B", "Hq", "Hkv", "hd"))
    lens, before = _lengths(case), _before(case)
    T = sum(lens)
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    st = dict(prefix_len=_whole(before), err=_whole([0] * B), longest=max(lens),
              cu_seqlens=None if max(lens) == 1 and min(lens) == 1 and case["op"] != "prompt" else _whole(ends))
    if case["op"] == "rotate" and not case["cache"]:
        blocks = 0
    else:
        blocks, table = _pages(case, seed)
        if case["op"] == "step" and case["window"]:  # pages that no query sees any more
            for b, p in enumerate(before):
                table[b, -(-case["sinks"] // PAGE):_first(case, p) // PAGE] = -1
        st["block_table"] = table.to(DEVICE)
    if case["op"] == "rotate":
        io = TYPES[case["io"]]
        whole = torch.cat([_normal(g, T, Hq * hd), _normal(g, T, Hkv * hd) * 2, _normal(g, T, Hkv * hd)], dim=1).to(io)
        q, k, v = whole.split([Hq * hd, Hkv * hd, Hkv * hd], dim=1)  # slices of one projection's output
        st.update(q=q.unflatten(1, (Hq, hd)), k=k.unflatten(1, (Hkv, hd)), v=v.unflatten(1, (Hkv, hd)) if blocks else None,
                  q_weight=(1 + 0.1 * _normal(g, hd)).to(io) if case["weight"] else None,
                  k_weight=(1 + 0.1 * _normal(g, hd)).to(io) if case["weight"] else None,
                  q_out=torch.zeros(T, Hq, hd, device=DEVICE, dtype=io), rotary=case["rotary"])
        if blocks:
            st.update({n: torch.zeros(blocks, Hkv, PAGE, hd, device=DEVICE, dtype=io) for n in ("k_cache", "v_cache")})
        else:
            st["k_out"] = torch.zeros(T, Hkv, hd, device=DEVICE, dtype=io)
        return st
    q = _normal(g, T, Hq, hd)
    st.update(q=(q * 1.5).to(torch.bfloat16), out=torch.zeros(T, Hq, hd, device=DEVICE, dtype=torch.bfloat16),
              window=case["window"], sinks=case["sinks"])
    st.update({n: torch.randn(blocks, Hkv, PAGE, hd, generator=g, device=DEVICE, dtype=torch.bfloat16)
               for n in ("k_cache", "v_cache")})
    if case["op"] == "step":
        st["live"] = _whole([int(x) for x in _live(case)]) if case["idle"] else None
        st["most"] = max(before) + 1
    else:  # the lengths, which the program that made the batch knows
        st["parts"] = list(zip(ends, lens, before))
    return st


def _drafts(case, g, seed):
    B, N, V, io = case["B"], case["N"], case["V"], TYPES[case["io"]]
    rng = random.Random(seed)
    shape = [[-1] + [i - 1 if case["shape"] == "chain" else rng.randint(max(0, i // 3 - 2), i - 1) for i in range(1, N)]
             for _ in range(B)]
    parents = _whole(shape)
    logits = 5 * torch.randn(B, N, V, generator=g, device=DEVICE, dtype=io)
    target = torch.softmax(logits, -1, dtype=torch.float32).to(io)
    # the draft has the target's opinion, more or less
    logits += torch.randn(B, N, V, generator=g, device=DEVICE, dtype=io)
    draft = torch.softmax(logits, -1, dtype=torch.float32).to(io)
    del logits
    at = parents.long().clamp(min=0)
    if case["known"]:
        # each node's token is drawn from the draft's probabilities at its parent
        tokens = torch.stack([torch.searchsorted(row.float().cumsum(-1), torch.rand(N, 1, generator=g, device=DEVICE) * 0.999)
                              .clamp(max=V - 1).gather(1, torch.zeros(N, 1, dtype=torch.long, device=DEVICE))[:, 0]
                              for row in (draft[b][at[b]] for b in range(B))])
    else:
        # the n-th child of a node is the draft's n-th token there
        places = _whole([[sum(p == row[i] for p in row[1:i]) for i in range(N)] for row in shape]).long()
        best = torch.topk(draft.float().flatten(0, 1), min(N, V)).indices.unflatten(0, (B, N))
        tokens = best.gather(1, at[..., None].expand(B, N, best.shape[-1])).gather(2, places[..., None])[..., 0]
        draft = None
    return dict(parents=parents, tokens=tokens.to(torch.int32), target=target, draft=draft,
                uniforms=torch.rand(B, N, generator=g, device=DEVICE), path=torch.zeros(B, N, device=DEVICE, dtype=torch.int32),
                length=_whole([0] * B), next=_whole([0] * B), err=_whole([0] * B))


def prepare(case, seed):
    return dict(_inputs(case, seed), op=case["op"])


def run(st):
    return {"rotate": _rotate, "prompt": _prompt, "step": _step, "accept": _accept}[st["op"]](st)


def _rotate(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_qk_norm_rope(st["q"], st["k"], st["q_out"], st["prefix_len"], st["err"], k_out=st.get("k_out"), v=st["v"],
                           k_cache=st.get("k_cache"), v_cache=st.get("v_cache"), block_table=st.get("block_table"),
                           cu_seqlens=st["cu_seqlens"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                           rotary_dim=st["rotary"], rope_theta=THETA)
        return {n: st[n] for n in ("q_out", "k_out", "k_cache", "v_cache") if n in st}
    T, rotary, before = st["q"].shape[0], st["rotary"], st["prefix_len"].long()
    token = torch.arange(T, device=before.device)
    if st["cu_seqlens"] is None:
        seq, position = token, before
    else:
        cu = st["cu_seqlens"].long()
        seq = torch.searchsorted(cu, token, right=True) - 1
        position = before[seq] + token - cu[seq]
    # far positions lose their angles in 32 bits
    turn = position.double()[:, None] * THETA ** (-torch.arange(0, rotary, 2, device=token.device).double() / rotary)
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * w.float() if w is not None else x
        a, b, rest = x.split([rotary // 2, rotary // 2, x.shape[-1] - rotary], dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1).to(st["q_out"].dtype)

    st["q_out"].copy_(turned(st["q"], st["q_weight"]))
    k = turned(st["k"], st["k_weight"])
    if "k_out" in st:
        st["k_out"].copy_(k)
        return {"q_out": st["q_out"], "k_out": st["k_out"]}
    block, row = st["block_table"].long()[seq, position // PAGE], position % PAGE
    st["k_cache"][block, :, row] = k
    st["v_cache"][block, :, row] = st["v"]
    return {n: st[n] for n in ("q_out", "k_cache", "v_cache")}


def _prompt(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_window_attn_prompt(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["cu_seqlens"],
                                 st["prefix_len"], st["out"], st["err"], window=st["window"], sinks=st["sinks"],
                                 max_len=st["longest"])
        return st["out"]
    Hq, hd = st["q"].shape[1:]
    Hkv, W, sinks = st["k_cache"].shape[1], st["window"], st["sinks"]
    # the scores of a long prompt do not fit at once: sequences, and parts of long ones, follow one another
    for b, (first, n, before) in enumerate(st["parts"]):
        most = max(1, PIECE // (4 * Hq * (before + n) or 1))
        for start in range(0, n, most):
            count = min(most, n - start)
            p = before + start
            lo = max(0, p - W + 1) if W else 0
            place = torch.cat([torch.arange(min(sinks, lo), device=st["q"].device),
                               torch.arange(lo, p + count, device=st["q"].device)])
            block = st["block_table"][b].long()[place // PAGE]
            k, v = (st[c][block, :, place % PAGE].float().transpose(0, 1)[:, None] for c in ("k_cache", "v_cache"))
            q = st["q"][first + start:first + start + count].float().unflatten(1, (Hkv, Hq // Hkv)).movedim(0, 2)
            scores = (q @ k.transpose(-1, -2)) * hd ** -0.5
            at = p + torch.arange(count, device=place.device)[:, None]
            seen = place <= at
            if W:
                seen &= (at - place < W) | (place < sinks)
            scores.masked_fill_(~seen, -math.inf)
            scores = torch.exp_(scores.sub_(scores.amax(-1, keepdim=True)))
            o = (scores @ v) / scores.sum(-1, keepdim=True)
            st["out"][first + start:first + start + count] = o.movedim(2, 0).flatten(1, 2).to(st["out"].dtype)
    return st["out"]


def _step(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_window_attn_step(st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["prefix_len"], st["out"],
                               st["err"], window=st["window"], sinks=st["sinks"], live=st["live"])
        return st["out"]
    Hq, hd = st["q"].shape[1:]
    Hkv, W, sinks, at = st["k_cache"].shape[1], st["window"], st["sinks"], st["prefix_len"].long()[:, None]
    if W:
        near = at - W + 1 + torch.arange(W, device=at.device)
        far = torch.arange(sinks, device=at.device).expand(at.shape[0], sinks)
        place = torch.cat([far, near], dim=1)
        seen = torch.cat([far < near[:, :1], near >= 0], dim=1)
    else:
        place = torch.arange(st["most"], device=at.device).expand(at.shape[0], -1)
        seen = place <= at
    place = torch.where(seen, place, at)
    block, row = st["block_table"].long().gather(1, place // PAGE), place % PAGE
    k, v = (st[c][block, :, row].float().transpose(1, 2)[:, :, None] for c in ("k_cache", "v_cache"))
    q = st["q"].float().unflatten(1, (Hkv, Hq // Hkv))[:, :, :, None]
    scores = (q @ k.transpose(-1, -2)) * hd ** -0.5
    scores = scores.masked_fill(~seen[:, None, None, None], -math.inf)
    scores = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = ((scores @ v) / scores.sum(-1, keepdim=True)).flatten(1, 4).unflatten(1, (Hq, hd)).to(st["out"].dtype)
    st["out"].copy_(o if st["live"] is None else torch.where(st["live"].bool()[:, None, None], o, st["out"]))
    return st["out"]


def _accept(st):
    if own:
        import tree_speculative_verification_gdn_gb300 as tv
        tv.tv_accept_sample(st["parents"], st["tokens"], st["target"], st["draft"], st["uniforms"], st["path"], st["length"],
                            st["next"], st["err"])
        return {"path": st["path"], "length": st["length"], "next": st["next"]}
    # A node is tested when its parent is the last accepted one; `left` is what the tokens refused there leave of
    # the target's probabilities.  64 bits: a token next to a border decides.
    parents, tokens, target, draft = st["parents"].long(), st["tokens"].long(), st["target"], st["draft"]
    B, N, V = target.shape
    u, every = st["uniforms"].double(), torch.arange(B, device=parents.device)
    node, count, mass = torch.zeros_like(every), torch.ones_like(every), torch.ones_like(u[:, 0])
    path = torch.full_like(st["path"], -1)
    path[:, 0] = 0
    left = target[:, 0].double()
    for i in range(1, N):
        tested, x = parents[:, i] == node, tokens[:, i]
        have = left[every, x]
        given = draft[every, node, x].double() if draft is not None else torch.ones_like(have)
        yes = tested & (u[:, i] * given * mass < have)
        no = tested & ~yes
        if draft is not None:
            less = (left - draft[every, node].double()).clamp(min=0)
            total = less.sum(-1, keepdim=True)
            less = torch.where(total > 0, less / total, target[every, node].double())
        else:
            less = left.clone()
            less[every, x] = 0
            mass = torch.where(no, mass - have, torch.where(yes, 1.0, mass))
        node = torch.where(yes, i, node)
        path[every, torch.where(yes, count, 0)] = torch.where(yes, i, 0).to(path.dtype)
        count = count + yes
        left = torch.where(yes[:, None], target[every, node].double(), torch.where(no[:, None], less, left))
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, target[every, node].double())
    sums = left.cumsum(-1)
    token = torch.searchsorted(sums, u[:, :1] * sums[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    return {"path": path, "length": count.to(torch.int32), "next": token.to(torch.int32)}


def exact(case, seed):
    """The definitions in 64 bits."""
    if case["op"] == "prompt" and _size(case) > 2 ** 40:
        return None
    st = _inputs(case, seed)
    if case["op"] == "accept":
        return _exact_accept(case, st)
    if case["op"] == "rotate":
        return _exact_rotate(case, st)
    B, Hq, Hkv, hd = (case[n] for n in ("B", "Hq", "Hkv", "hd"))
    out = torch.zeros(sum(_lengths(case)), Hq, hd, device=DEVICE, dtype=torch.float64)
    t = 0
    for b, (p, n) in enumerate(zip(_before(case), _lengths(case))):
        if case["op"] == "step" and not _live(case)[b]:
            t += n
            continue
        table = st["block_table"][b].tolist()
        lo = _first(case, p)
        hidden = set(range(-(-min(case["sinks"], lo) // PAGE), lo // PAGE))
        pages = [0 if i in hidden else max(x, 0) for i, x in enumerate(table[:-(-(p + n) // PAGE)])]
        keys, values = (torch.zeros(Hkv, 0, hd) if not pages else
                        st[c][torch.tensor(pages, device=DEVICE)].transpose(0, 1).reshape(Hkv, -1, hd)[:, :p + n]
                        for c in ("k_cache", "v_cache"))
        for h in range(Hq):
            for a in range(0, n, 4096):
                m = min(4096, n - a)
                z = _first(case, p + a) if case["window"] else 0
                z = max(z, min(case["sinks"], z))
                i = torch.cat([torch.arange(min(case["sinks"], z), device=DEVICE), torch.arange(z, p + a + m, device=DEVICE)])
                kk, vv = (x[h // (Hq // Hkv)][i].double() for x in (keys, values))
                j = torch.arange(p + a, p + a + m, device=DEVICE)
                away = j[:, None] - i[None]
                hide = away < 0
                if case["window"]:
                    hide |= (away >= case["window"]) & (i[None] >= case["sinks"])
                s = torch.einsum("td,kd->tk", st["q"][t + a:t + a + m, h].double(), kk) / math.sqrt(hd)
                out[t + a:t + a + m, h] = torch.softmax(s.masked_fill(hide, -math.inf), dim=1) @ vv
        t += n
    return out


def _exact_rotate(case, st):
    hd, half = case["hd"], case["rotary"] // 2
    position = torch.cat([torch.arange(p, p + n, dtype=torch.float64) for p, n in zip(_before(case), _lengths(case))])
    angle = position[:, None] / THETA ** (torch.arange(half, dtype=torch.float64) * 2 / case["rotary"])
    spin = torch.polar(torch.ones_like(angle), angle).to(DEVICE)[:, None]
    got = {}
    for name in ("q", "k"):
        x = st[name].double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / hd + EPS)
        if st[name + "_weight"] is not None:
            x = x * st[name + "_weight"].double()
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * spin
        got[name] = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
    if "k_out" in st:
        return {"q_out": got["q"], "k_out": got["k"]}
    caches = {n: torch.zeros(st[n].shape, device=DEVICE, dtype=torch.float64) for n in ("k_cache", "v_cache")}
    t = 0
    for b, (p, n) in enumerate(zip(_before(case), _lengths(case))):
        pos = torch.arange(p, p + n, device=DEVICE)
        block = st["block_table"][b].long()[pos // PAGE]
        caches["k_cache"][block, :, pos % PAGE] = got["k"][t:t + n]
        caches["v_cache"][block, :, pos % PAGE] = st["v"][t:t + n].double()
        t += n
    return {"q_out": got["q"], **caches}


def _exact_accept(case, st):
    B, N = case["B"], case["N"]
    path, length, token = torch.full((B, N), -1, dtype=torch.int32), torch.ones(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        parents, tokens, u = (st[n][b].tolist() for n in ("parents", "tokens", "uniforms"))
        node, walked = 0, [0]
        while True:
            p = st["target"][b, node].double()
            q = None if st["draft"] is None else st["draft"][b, node].double()
            r, mass, went = p.clone(), 1.0, None
            for c in range(node + 1, N):
                if parents[c] != node:
                    continue
                x = tokens[c]
                if u[c] * mass * (1.0 if q is None else q[x].item()) < r[x].item():
                    went = c
                    break
                if q is None:
                    mass -= r[x].item()
                    r[x] = 0
                else:
                    r = torch.relu(r - q)
                    r = r / r.sum() if r.sum().item() > 0 else p.clone()
            if went is None:
                break
            node = went
            walked.append(node)
        if r.sum().item() == 0:
            r = p
        sums = torch.cumsum(r, 0)
        token[b] = min(int((sums <= u[0] * sums[-1]).sum()), case["V"] - 1)
        path[b, :len(walked)] = torch.tensor(walked, dtype=torch.int32)
        length[b] = len(walked)
    return {"path": path, "length": length, "next": token}
