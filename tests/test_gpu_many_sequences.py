"""Thousands of packed sequences, most of them empty: the lengths are read by every block of the check up to 1024
sequences, by one block first past that."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import BF, DEV, attend, case, check, whole
from test_gpu_qk_rope import cached, make, near, positions

pytestmark = pytest.mark.gpu


def some(B, seed):
    """Lengths and prefixes of B sequences, about 600 of them with tokens, the last among them."""
    rng = np.random.default_rng(seed)
    lens = np.where(rng.random(B) < 600 / B, rng.integers(1, 4, size=B), 0)
    lens[-1] = 2
    return lens.tolist(), rng.integers(0, 30, size=B).tolist()


def table_of(lens, prefix, seed):
    """A page for each sixteen tokens of a sequence that has any; entries of no page lie outside the cache."""
    needs = [-(-(p + n) // 16) if n else 0 for p, n in zip(prefix, lens)]
    blocks = sum(needs) + 2
    order = iter(np.random.default_rng(seed).permutation(blocks).tolist())
    table = np.full((len(lens), 3), 1 << 30, dtype=np.int32)
    for b, n in enumerate(needs):
        table[b, :n] = [next(order) for _ in range(n)]
    return blocks, table


@pytest.mark.parametrize("B", [1023, 1024, 1025, 2048, 2049, 9001])
def test_rotation(B):
    lens, prefix = some(B, B)
    c = make(lens, 2, 1, 64, seed=B)
    blocks, table = table_of(lens, prefix, B)
    bad = next(b for b in range(B // 2, B) if lens[b])
    table[bad, (prefix[bad] + lens[bad] - 1) // 16] = -5
    live = np.ones(B)
    idle = next(b for b in range(B) if lens[b])
    live[idle] = 0
    q, kc, vc, err = cached(c, prefix, table, blocks, rotary=64, live=whole(live))
    assert err == [tv.TV_ERR_BAD_BLOCK if b == bad else 0 for b in range(B)]
    at, seq = positions(prefix, lens), np.repeat(np.arange(B), lens)
    there = (seq != bad) & (seq != idle)
    near(q[there], c["q"][there], c["qw"], at[there], 64, 1e4)
    assert (q[~there] == 7).all()
    block, row = torch.tensor(table[seq, at // 16], device=DEV)[there].long(), torch.tensor(at % 16, device=DEV)[there].long()
    near(kc[block, :, row], c["k"][there], c["kw"], at[there], 64, 1e4)
    assert torch.equal(vc[block, :, row], c["v"][there])
    vc[block, :, row] = 5.0
    assert (vc == 5).all()
    for cu in (np.r_[0, np.cumsum(lens)[:-1], np.sum(lens) + 1], np.r_[0, np.cumsum(lens)[:-1], np.sum(lens) - 3]):
        c["cu"] = whole(cu)
        q, kc, vc, err = cached(c, prefix, table, blocks, rotary=64)
        assert err == [tv.TV_ERR_BAD_SEQLEN] * B and (q == 7).all() and (kc == 5).all() and (vc == 5).all()


@pytest.mark.parametrize("B", [1024, 1025, 5003])
@pytest.mark.parametrize("max_len", [3, 40])              # few query rows, and tiles of them
def test_attention(B, max_len):
    lens, prefix = some(B, B)
    c = case(lens, prefix, 2, 1, 64, seed=B)
    out, err = attend(c, window=9, sinks=2, max_len=max_len)
    assert not any(err)
    check(c, out, 9, 2)
    out, err = attend(c, window=9, sinks=2, max_len=1)
    assert err == [tv.TV_ERR_BAD_SEQLEN] * B and (out == 7).all()


def test_time_grows_with_their_number_not_its_square():
    # eight times the sequences, the same tokens: eight times the time at most, but for what a launch takes
    def time_of(B):
        lens = [1] * 512 + [0] * (B - 512)
        cu, prefix, err = whole(np.r_[0, np.cumsum(lens)]), whole(np.zeros(B)), whole(np.full(B, 9))
        table = whole(np.minimum(np.arange(B), 511)[:, None])
        q, k, v = (torch.randn(512, 1, 64, device=DEV).to(BF) for _ in range(3))
        kc, vc = (torch.zeros(512, 1, 16, 64, device=DEV, dtype=BF) for _ in range(2))
        out, times = torch.empty_like(q), []
        for _ in range(4):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            tv.tv_qk_norm_rope(q, k, out, prefix, err, v=v, k_cache=kc, v_cache=vc, block_table=table, cu_seqlens=cu)
            tv.tv_window_attn_prompt(out, kc, vc, table, cu, prefix, torch.empty_like(q), err, max_len=1)
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        assert not err.any()
        return min(times)
    few, many = time_of(1 << 15), time_of(1 << 18)
    assert many <= 16 * few, (few, many)
