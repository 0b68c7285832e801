"""Acceptance by probabilities against the fp64 oracle: paths, lengths and tokens are equal.  Random numbers are
multiples of 2^-24 and sums are good to 2^-44, so that of some thousand draws none lies between."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from oracle import window as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, N, V, io="f32", shape="tree", known=True, seed=0, sharp=3.0, noise=1.0):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    parents = np.array([[-1] + [i - 1 if shape == "chain" else 0 if shape == "star" else int(rng.integers(max(0, i // 3 - 1), i))
                                for i in range(1, N)] for _ in range(B)])
    logits = sharp * torch.randn(B, N, V, generator=g)
    target = torch.softmax(logits, -1).to(TYPES[io])
    draft = torch.softmax(logits + noise * torch.randn(B, N, V, generator=g), -1).to(TYPES[io])
    tokens = np.zeros((B, N), dtype=np.int64)
    for b in range(B):
        for i in range(1, N):
            p = parents[b, i]
            if known:
                w = draft[b, p].double().numpy()
                tokens[b, i] = min(np.searchsorted(np.cumsum(w) / w.sum(), rng.random()), V - 1)
            else:
                place = int((parents[b, 1:i] == p).sum())
                tokens[b, i] = int(torch.topk(target[b, p].float(), min(place + 1, V)).indices[-1])
    return dict(parents=parents, tokens=tokens, target=target, draft=draft if known else None,
                u=torch.rand(B, N, generator=g))


def accept(c, Lmax=None, stream=None):
    B, N, V = c["target"].shape
    Lmax = N if Lmax is None else Lmax
    dev = [torch.as_tensor(np.asarray(c[n]), dtype=torch.int32, device=DEV) for n in ("parents", "tokens")]
    dev += [c["target"].to(DEV), None if c["draft"] is None else c["draft"].to(DEV), c["u"].float().to(DEV)]
    out = [torch.full(s, 777, dtype=torch.int32, device=DEV) for s in ((B, Lmax), (B,), (B,), (B,))]
    torch.cuda.synchronize()
    tv.tv_accept_sample(*dev, *out, stream=stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in out]


def check(c, got, Lmax=None):
    path, length, token, err = got
    B, N, V = c["target"].shape
    for b in range(B):
        want = O.accept_sample(c["parents"][b], c["tokens"][b], c["target"][b].double().numpy(),
                               None if c["draft"] is None else c["draft"][b].double().numpy(), c["u"][b].numpy(),
                               N if Lmax is None else Lmax)
        assert err[b] == 0
        assert path[b, :length[b]].tolist() == want[0] and (path[b, length[b]:] == -1).all(), b
        assert token[b] == want[1], b


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("shape", ["chain", "tree", "star"])
def test_trees(io, known, shape):
    for seed in range(4):
        c = make(8, 9, 1000 + seed, io, shape, known, seed)
        check(c, accept(c))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 31, 127, 513, 4097, 16001, 50021])
def test_vocabularies(io, known, V):
    c = make(4, 4, V, io, "star" if V % 2 else "chain", known, seed=V, noise=2.0)
    check(c, accept(c))


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 100, 256])
def test_numbers_of_nodes(N):
    for known, sharp in ((True, 2.0), (False, 4.0)):
        c = make(3, N, 300, "f32", "tree", known, seed=N, sharp=sharp)
        check(c, accept(c))


@pytest.mark.parametrize("Lmax", [1, 2, 3, 40])
def test_room_for_the_path(Lmax):
    c = make(6, 12, 64, "f32", "chain", True, seed=1, noise=0.3)
    check(c, accept(c, Lmax), Lmax)


def test_many_refusals_in_a_row():
    # the draft is nearly disjoint from the target: each refusal goes through the residual of the one before
    c = make(16, 24, 600, "f32", "star", True, seed=2, noise=6.0)
    got = accept(c)
    check(c, got)
    c = make(16, 24, 600, "f32", "star", False, seed=3, sharp=0.1)
    got = accept(c)
    check(c, got)
    assert (got[1] == 1).any()


def test_batch_and_a_long_row():
    c = make(200, 3, 700, "f32", "chain", True, seed=4)
    check(c, accept(c))
    c = make(2, 3, 400_003, "bf16", "star", True, seed=5, noise=2.0)
    check(c, accept(c))


def test_borders_are_exact():
    # probabilities in 32nds and random numbers on their borders: u = 4/32 is the second token's, not the first's
    p = torch.zeros(33, 1, 8)
    p[:, 0] = torch.tensor([4, 0, 12, 8, 0, 4, 4, 0]) / 32.0
    u = torch.arange(33)[:, None] / 32.0
    c = dict(parents=[[-1]] * 33, tokens=[[0]] * 33, target=p, draft=None, u=u)
    token = accept(c)[2].tolist()
    assert token == [0] * 4 + [2] * 12 + [3] * 8 + [5] * 4 + [6] * 4 + [6]      # a number of 1: the last one with any
    # acceptance: u q < p, so u = p / q refuses
    t = torch.tensor([[0.25, 0.75], [0.5, 0.5]])
    q = torch.tensor([[0.5, 0.5], [0.5, 0.5]])
    c = dict(parents=[[-1, 0]] * 2, tokens=[[0, 0]] * 2, target=torch.stack([t, t]), draft=torch.stack([q, q]),
             u=torch.tensor([[0.0, 0.5], [0.0, 0.5 - 2.0 ** -24]]))
    path, length, token, err = accept(c)
    assert length.tolist() == [1, 2] and token.tolist() == [1, 0] and not err.any()


def test_equal_distributions_are_never_refused():
    c = make(32, 6, 500, "f32", "chain", True, seed=6)
    c["draft"] = c["target"].clone()
    rng = np.random.default_rng(0)
    for b in range(32):
        for i in range(1, 6):
            w = c["target"][b, i - 1].double().numpy()
            c["tokens"][b, i] = np.searchsorted(np.cumsum(w) / w.sum(), rng.random())
    got = accept(c)
    assert (got[1] == 6).all()
    check(c, got)


def test_residual_of_nothing_starts_again_from_the_target():
    # p = q and a token without a probability: refused, and p - q leaves nothing
    p = torch.tensor([0.5, 0.5, 0.0, 0.0])
    t = p.expand(1, 3, 4).contiguous()
    c = dict(parents=[[-1, 0, 0]], tokens=[[0, 2, 1]], target=t, draft=t, u=torch.tensor([[0.7, 0.0, 0.9]]))
    got = accept(c)
    assert got[0].tolist() == [[0, 2, -1]] and got[2].tolist() == [1]
    check(c, got)
    # every token refused by hand: the draw is the target's
    t = torch.tensor([1.0, 0.0]).expand(1, 2, 2).contiguous()
    c = dict(parents=[[-1, 0]], tokens=[[0, 0]], target=t, draft=None, u=torch.tensor([[0.5, 1.0]]))
    got = accept(c)
    assert got[1].tolist() == [1] and got[2].tolist() == [0]


def test_tokens_out_of_range_twice_the_same_and_odd_probabilities():
    c = make(4, 6, 50, "f32", "star", False, seed=7, sharp=0.5)
    c["tokens"][:, 1], c["tokens"][:, 2], c["tokens"][:, 4] = -1, 50, c["tokens"][:, 3]
    check(c, accept(c))
    c = make(4, 6, 50, "f32", "star", True, seed=8)
    c["tokens"][:, 1], c["tokens"][:, 2] = 1 << 30, -(1 << 30)
    c["target"][:, :, 3], c["target"][:, :, 4], c["draft"][:, :, 5] = -1.0, float("nan"), float("nan")
    c["tokens"][:, 3], c["tokens"][:, 4] = 3, 4
    check(c, accept(c))


def test_errors_are_reported():
    c = make(4, 5, 40, seed=9)
    c["parents"][1, 2] = 2
    c["parents"][2, 3] = -2
    c["target"][3] = 0.0
    path, length, token, err = accept(c, 3)
    assert err.tolist() == [0, tv.TV_ERR_BAD_TREE, tv.TV_ERR_BAD_TREE, tv.TV_ERR_BAD_PROBS]
    assert (path[1:] == -1).all() and length[1:].tolist() == [0] * 3 and token[1:].tolist() == [-1] * 3
    for bad in (float("inf"), float("nan")):
        c = make(2, 3, 40, seed=10)
        c["target"][0] = bad
        path, length, token, err = accept(c)
        assert err[1] == 0 and err[0] in (0, tv.TV_ERR_BAD_PROBS) and -1 <= token[0] < 40


def test_same_results_every_time_on_any_stream_and_in_a_graph():
    c = make(20, 8, 9000, "f32", "tree", True, seed=11, noise=2.0)
    a = accept(c)
    side = torch.cuda.Stream()
    b = accept(c, stream=side)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    dev = [torch.as_tensor(np.asarray(c[n]), dtype=torch.int32, device=DEV) for n in ("parents", "tokens")]
    dev += [c["target"].to(DEV), c["draft"].to(DEV), c["u"].to(DEV)]
    out = [torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((20, 8), (20,), (20,), (20,))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.tv_accept_sample(*dev, *out)
    for seed in (0, 1):
        c["u"] = torch.rand(20, 8, generator=torch.Generator().manual_seed(seed))
        dev[4].copy_(c["u"])
        graph.replay()
        torch.cuda.synchronize()
        check(c, [x.cpu().numpy() for x in out])


def test_counts_follow_the_target():
    # one token after another over 4096 sequences of the same probabilities
    B, V = 4096, 6
    p = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05, 0.0])
    q = torch.tensor([0.1, 0.2, 0.3, 0.1, 0.1, 0.2])
    g = torch.Generator().manual_seed(12)
    tokens = torch.stack([torch.zeros(B, dtype=torch.long)] + [torch.multinomial(q, B, True, generator=g) for _ in range(2)], 1)
    c = dict(parents=[[-1, 0, 0]] * B, tokens=tokens.numpy(), target=p.expand(B, 3, V).contiguous(),
             draft=q.expand(B, 3, V).contiguous(), u=torch.rand(B, 3, generator=g))
    path, length, token, err = accept(c)
    first = np.where(length == 1, token, tokens.numpy()[np.arange(B), np.where(length > 1, path[:, 1], 0)])
    # counts of 4096 draws: five standard deviations
    count = np.bincount(first, minlength=V) / B
    assert (np.abs(count - p.numpy()) <= 5 * np.sqrt(p.numpy() * (1 - p.numpy()) / B) + 1e-12).all(), count
