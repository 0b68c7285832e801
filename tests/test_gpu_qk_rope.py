"""Norms of queries and keys with their rotation, into dense outputs and the paged cache, against the fp64 oracle.

Bounds, per element, u = 2^-24: a mean of squares over hd columns in 16-term chains (20 u), its root (half of that, and
4 u), two products and a sum for weight and scale (4 u): 19 u of |y|; a rotation with cosines off by 3 u and three
roundings: 25 u (|a| + |b|) of a pair; 32 allowed.  A bf16 result is rounded once: 2^-8 of it."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import BF, DEV, U, f64, pages, whole
from oracle import window as O

pytestmark = pytest.mark.gpu
TYPES = {"bf16": BF, "f32": torch.float32}
EPS = 1e-6


def make(lens, Hq, Hkv, hd, io="bf16", seed=0, fused=True):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    x = torch.randn(T, (Hq + 2 * Hkv) * hd, generator=g).to(TYPES[io]).to(DEV)
    parts = [p.unflatten(1, (n, hd)) for p, n in zip(x.split([Hq * hd, Hkv * hd, Hkv * hd], dim=1), (Hq, Hkv, Hkv))]
    if not fused:
        parts = [p.contiguous() for p in parts]
    qw, kw = ((1 + 0.2 * torch.randn(hd, generator=g)).to(TYPES[io]).to(DEV) for _ in range(2))
    return dict(q=parts[0], k=parts[1], v=parts[2], qw=qw, kw=kw, cu=whole(np.concatenate([[0], np.cumsum(lens)])), lens=lens)


def near(got, x, weight, positions, rotary, theta, norm=True, offset=0.0):
    x = f64(x)
    y = O.norm_rotate(x, None if weight is None else f64(weight), positions, rotary, theta, EPS, norm, offset)
    n = O.norm_rotate(x, None if weight is None else f64(weight), positions, 0, theta, EPS, norm, offset)
    size, half = np.abs(n), rotary // 2
    size[..., :half] += np.abs(n[..., half:rotary])
    size[..., half:rotary] = size[..., :half]
    tol = 32 * U * size + (2.0 ** -8 * np.abs(y) if got.dtype == BF else 0.0)
    over = np.abs(f64(got) - y) - tol
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} past the bound, worst by {over.max():.3e}"


def positions(prefix, lens):
    return np.concatenate([np.arange(p, p + n) for p, n in zip(prefix, lens)])


def dense(c, prefix, rotary, theta=1e4, cu=True, weights=True, **more):
    q_out, k_out = torch.full_like(c["q"], 7.0).contiguous(), torch.full_like(c["k"], 7.0).contiguous()
    err = torch.full((len(c["lens"]),), 9, dtype=torch.int32, device=DEV)
    tv.tv_qk_norm_rope(c["q"], c["k"], q_out, None if prefix is None else whole(prefix), err, k_out=k_out,
                       cu_seqlens=c["cu"] if cu else None, q_weight=c["qw"] if weights else None,
                       k_weight=c["kw"] if weights else None, eps=EPS, rotary_dim=rotary, rope_theta=theta, **more)
    torch.cuda.synchronize()
    return q_out, k_out, err.tolist()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hd,rotary", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 32), (128, 112), (256, 256), (256, 64), (256, 0)])
def test_types_heads_and_rotations(io, hd, rotary):
    lens, prefix = [37, 0, 1, 20], [0, 9, 1000, 65535]
    c = make(lens, 6, 2, hd, io, seed=hd + rotary)
    at = positions(prefix, lens)
    q, k, err = dense(c, prefix, rotary)
    assert err == [0] * 4
    near(q, c["q"], c["qw"], at, rotary, 1e4)
    near(k, c["k"], c["kw"], at, rotary, 1e4)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (16, 4), (64, 8), (96, 96)])
def test_numbers_of_heads(io, Hq, Hkv):
    for lens in ([1], [2] * 3, [50]):
        c = make(lens, Hq, Hkv, 128, io, seed=Hq, fused=False)
        at = positions([3] * len(lens), lens)
        q, k, err = dense(c, [3] * len(lens), 128, theta=1e6, weights=False)
        assert not any(err)
        near(q, c["q"], None, at, 128, 1e6)
        near(k, c["k"], None, at, 128, 1e6)


@pytest.mark.parametrize("theta", [1.0, 1e4, 1e7])
def test_far_positions(theta):
    lens, prefix = [3] * 5, [0, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) - 5]
    c = make(lens, 2, 1, 128, "f32", seed=3)
    q, k, err = dense(c, prefix, 128, theta=theta)
    assert not any(err)
    # the oracle's own angle is a product of 64 bits: 2^30 radians to 2^-23; the bound allows as much at the far end
    for (a, b), p in zip(((0, 3), (3, 6), (6, 9), (9, 12)), prefix):
        near(q[a:b], c["q"][a:b], c["qw"], np.arange(p, p + 3), 128, theta)
        near(k[a:b], c["k"][a:b], c["kw"], np.arange(p, p + 3), 128, theta)


def test_one_token_each_offset_no_norm_and_rows_in_place():
    c = make([1] * 9, 4, 2, 128, seed=4)
    prefix = [0, 1, 15, 16, 17, 100, 2, 3, 4]
    q, k, err = dense(c, prefix, 128, cu=False, weight_offset=1.0)
    assert not any(err)
    near(q, c["q"], c["qw"], prefix, 128, 1e4, offset=1.0)
    near(k, c["k"], c["kw"], prefix, 128, 1e4, offset=1.0)
    q, k, err = dense(c, prefix, 64, cu=False, norm=False, weights=False)
    near(q, c["q"], None, prefix, 64, 1e4, norm=False)
    near(k, c["k"], None, prefix, 64, 1e4, norm=False)
    want, _, _ = dense(c, None, 0, cu=False)
    near(want, c["q"], c["qw"], [0] * 9, 0, 1e4)
    mine = dict(c, q=c["q"].clone(), k=c["k"].clone())
    err = torch.zeros(9, dtype=torch.int32, device=DEV)
    tv.tv_qk_norm_rope(mine["q"], mine["k"], mine["q"], whole(prefix), err, k_out=mine["k"], q_weight=c["qw"], k_weight=c["kw"],
                       eps=EPS)
    a, b, _ = dense(c, prefix, 128, cu=False)
    torch.cuda.synchronize()
    assert torch.equal(mine["q"], a) and torch.equal(mine["k"], b)


def cached(c, prefix, table, blocks, cu=True, rotary=128, live=None, k_out=None):
    T, Hkv, hd = c["k"].shape
    kc, vc = (torch.full((blocks, Hkv, 16, hd), 5.0, dtype=BF, device=DEV) for _ in range(2))
    q_out = torch.full_like(c["q"], 7.0).contiguous()
    err = torch.full((len(c["lens"]),), 9, dtype=torch.int32, device=DEV)
    tv.tv_qk_norm_rope(c["q"], c["k"], q_out, whole(prefix), err, v=c["v"], k_cache=kc, v_cache=vc, block_table=whole(table),
                       cu_seqlens=c["cu"] if cu else None, q_weight=c["qw"], k_weight=c["kw"], eps=EPS, rotary_dim=rotary,
                       live=live, k_out=k_out)
    torch.cuda.synchronize()
    return q_out, kc, vc, err.tolist()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("lens,prefix", [([1], [0]), ([17, 0, 100, 3], [0, 4, 30, 15]), ([1] * 40, list(range(40)))])
def test_cache_holds_the_keys_and_values_and_nothing_else(hd, lens, prefix):
    c = make(lens, 8, 4, hd, seed=hd)
    blocks, table = pages([p + n for p, n in zip(prefix, lens)], hd)
    for cu in (True, False) if set(lens) == {1} else (True,):
        k_out = torch.zeros_like(c["k"]).contiguous()
        q, kc, vc, err = cached(c, prefix, table, blocks, cu, rotary=hd // 2, k_out=k_out)
        assert not any(err)
        at = positions(prefix, lens)
        near(q, c["q"], c["qw"], at, hd // 2, 1e4)
        seq = np.repeat(np.arange(len(lens)), lens)
        block, row = torch.tensor(table[seq, at // 16], device=DEV).long(), torch.tensor(at % 16, device=DEV).long()
        near(kc[block, :, row], c["k"], c["kw"], at, hd // 2, 1e4)
        assert torch.equal(kc[block, :, row], k_out) and torch.equal(vc[block, :, row], c["v"])
        kc[block, :, row] = 5.0
        vc[block, :, row] = 5.0
        assert (kc == 5).all() and (vc == 5).all()


@pytest.mark.parametrize("cu", [True, False])
def test_bad_and_idle_sequences_leave_everything_alone(cu):
    c = make([1] * 6, 4, 2, 128, seed=5)
    blocks, table = pages([40] * 6, 5, most=3)
    table[1, 1] = -1
    table[2, 1] = blocks
    table[5, 1] = -7                       # of a row that holds no sequence
    prefix = [20, 20, 20, 48, -1, 20]
    q, kc, vc, err = cached(c, prefix, table, blocks, cu, live=whole([1, 1, 1, 1, 1, 0]))
    assert err == [0] + [tv.TV_ERR_BAD_BLOCK] * 2 + [tv.TV_ERR_CAPACITY] * 2 + [0]
    assert (q[1:] == 7).all()
    near(q[:1], c["q"][:1], c["qw"], [20], 128, 1e4)
    kc[int(table[0, 1]), :, 4] = 5.0
    vc[int(table[0, 1]), :, 4] = 5.0
    assert (kc == 5).all() and (vc == 5).all()


def test_only_the_blocks_of_new_tokens_matter():
    c = make([3], 2, 1, 64, seed=6)
    blocks, table = pages([100], 6)
    table[0, :5] = -1                      # given back: behind a window
    q, kc, vc, err = cached(c, [90], table, blocks, rotary=64)
    assert err == [0]


@pytest.mark.parametrize("cu", [[0, 20, 10], [0, 20, 99], [-1, 20, 30], [5, 0, 30]])
def test_bad_lengths(cu):
    c = make([20, 10], 2, 1, 64, seed=7)
    c["cu"] = whole(cu)
    q, k, err = dense(c, [0, 0], 64)
    assert err == [tv.TV_ERR_BAD_SEQLEN] * 2 and (q == 7).all() and (k == 7).all()


def test_rows_of_no_sequence():
    c = make([30, 40], 3, 1, 64, seed=8)
    c["cu"] = whole([7, 30, 50])
    q, k, err = dense(c, [0, 100], 64)
    assert not any(err) and (q[:7] == 7).all() and (q[50:] == 7).all() and (k[:7] == 7).all() and (k[50:] == 7).all()
    at = np.concatenate([np.arange(23), np.arange(100, 120)])
    near(q[7:50], c["q"][7:50], c["qw"], at, 64, 1e4)
    c["cu"] = whole([0, 0, 0])
    q, k, err = dense(c, [0, 0], 64)
    assert not any(err) and (q == 7).all()


@pytest.mark.parametrize("Hq,Hkv,hd", [(4, 1, 64), (16, 4, 128), (8, 2, 256)])
def test_many_tokens_and_sequences(Hq, Hkv, hd):
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 90, size=150).tolist()
    prefix = rng.integers(0, 5000, size=150).tolist()
    c = make(lens, Hq, Hkv, hd, seed=9)
    blocks, table = pages([p + n for p, n in zip(prefix, lens)], 9)
    q, kc, vc, err = cached(c, prefix, table, blocks, rotary=hd)
    assert not any(err)
    at, seq = positions(prefix, lens), np.repeat(np.arange(150), lens)
    near(q, c["q"], c["qw"], at, hd, 1e4)
    block, row = torch.tensor(table[seq, at // 16], device=DEV).long(), torch.tensor(at % 16, device=DEV).long()
    near(kc[block, :, row], c["k"], c["kw"], at, hd, 1e4)
    assert torch.equal(vc[block, :, row], c["v"])


def test_rotation_agrees_with_the_tree_attentions():
    # keys that tv_tree_attn writes for a chain are those that this call writes for its positions
    import _gpu
    import workloads as W
    t = W.attn_case([[-1, 0, 1, 2]], [37], Hq=4, Hkv=2, hd=64, seed=0)
    res = _gpu.run_attn(t)
    blocks = t.k_cache.shape[0]
    kc, vc = t.k_cache.to(DEV), t.v_cache.to(DEV)
    q, k, v = (x[0].to(DEV) for x in (t.q, t.k_new, t.v_new))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tv.tv_qk_norm_rope(q, k, torch.empty_like(q), t.prefix_len.to(DEV), err, v=v, k_cache=kc, v_cache=vc,
                       block_table=t.block_table.to(DEV), cu_seqlens=whole([0, 4]), norm=False, rope_theta=t.rope_theta)
    torch.cuda.synchronize()
    assert err.tolist() == [0] and blocks == kc.shape[0]
    assert torch.equal(vc.cpu(), torch.as_tensor(res["v_cache"]).cpu())
    diff = (kc.float().cpu() - torch.as_tensor(res["k_cache"]).float().cpu()).abs()
    assert (diff <= 2.0 ** -7 * kc.float().cpu().abs() + 1e-6).all()     # a rounding of bf16 apart at most


def test_a_graph_and_another_stream():
    c = make([1] * 4, 4, 2, 128, seed=11)
    prefix = whole([5, 6, 7, 8])
    blocks, table = pages([64] * 4, 11)
    kc, vc = (torch.zeros(blocks, 2, 16, 128, dtype=BF, device=DEV) for _ in range(2))
    q_out, err, tab = torch.zeros_like(c["q"]).contiguous(), whole([9] * 4), whole(table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tv.tv_qk_norm_rope(c["q"], c["k"], q_out, prefix, err, v=c["v"], k_cache=kc, v_cache=vc, block_table=tab,
                           q_weight=c["qw"], k_weight=c["kw"], eps=EPS)
    for at in ([5, 6, 7, 8], [30, 31, 32, 33]):
        prefix.copy_(whole(at))
        graph.replay()
        torch.cuda.synchronize()
        assert err.tolist() == [0] * 4
        near(q_out, c["q"], c["qw"], at, 128, 1e4)
        for b, p in enumerate(at):
            near(kc[int(table[b, p // 16]), :, p % 16][None], c["k"][b:b + 1], c["kw"], [p], 128, 1e4)
