"""Windowed attention over the paged cache against the fp64 oracle: prompts, drafted chains, single tokens.  Slots that
no query sees hold NaN, and pages that none sees have left the table."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_gdn_gb300 as tv
from _window import BF, DEV, attend, case, check, f64, oracle, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (8, 2), (10, 2), (16, 1)])
def test_prompt_heads(hd, Hq, Hkv):
    c = case([37, 0, 1, 130], [0, 5, 17, 100], Hq, Hkv, hd, seed=hd + Hq)
    out, err = attend(c)
    assert err == [0] * 4
    check(c, out, 0, 0)


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (100, 2), (66, 1)])
def test_many_heads_on_one_key_head(Hq, Hkv):
    c = case([3, 2], [40, 0], Hq, Hkv, 128, seed=Hq)
    out, err = attend(c)
    assert err == [0, 0]
    check(c, out, 0, 0)
    c = case([1, 1], [40, 0], Hq, Hkv, 64, seed=Hq, step=True)
    out, err = attend(c, window=9)
    assert err == [0, 0]
    check(c, out, 9, 0)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [2, 15, 16, 17], [127, 128, 129], [255, 256, 257], [0, 0, 3], [5, 0], [600]])
def test_prompt_lengths(hd, lens):
    c = case(lens, [0] * len(lens), 4, 2, hd, seed=sum(lens))
    out, err = attend(c, max_len=max(lens))
    assert not any(err)
    check(c, out, 0, 0)


WINDOWS = [(1, 0), (1, 1), (16, 0), (17, 16), (100, 4), (128, 17), (300, 1), (5, 200), (50, 1000), (1000, 3)]


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_prompt_windows(hd, window, sinks):
    lens, prefix = [190, 3, 40], [0, 700, 333]
    unseen = [(b, min(sinks, max(0, p - window + 1)), max(0, p - window + 1)) for b, p in enumerate(prefix)]
    c = case(lens, prefix, 6, 2, hd, seed=window + sinks, unseen=unseen)
    out, err = attend(c, window, sinks)
    assert not any(err)
    check(c, out, window, sinks)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0)] + WINDOWS)
def test_step_windows(hd, window, sinks):
    prefix = [0, 1, 15, 16, 17, 127, 128, 300, 700, 1023]
    unseen = [] if not window else [(b, min(sinks, max(0, p - window + 1)), max(0, p - window + 1)) for b, p in enumerate(prefix)]
    c = case([1] * len(prefix), prefix, 8, 2, hd, seed=window + sinks, unseen=unseen, step=True)
    out, err = attend(c, window, sinks)
    assert not any(err)
    check(c, out, window, sinks)


@pytest.mark.parametrize("hd,Hq,Hkv", [(128, 4, 1), (64, 5, 5), (256, 16, 1), (128, 24, 1)])
def test_step_long_context_few_sequences(hd, Hq, Hkv):
    # far more keys than sequences and heads: the keys are spread over many SMs and joined
    c = case([1, 1], [5000, 77], Hq, Hkv, hd, seed=hd, step=True)
    out, err = attend(c)
    assert not any(err)
    check(c, out, 0, 0)
    again, _ = attend(c)
    assert torch.equal(out, again)


@pytest.mark.parametrize("hd,Hq,Hkv", [(128, 4, 1), (64, 6, 2), (256, 8, 2), (128, 32, 1)])
@pytest.mark.parametrize("n", [2, 5, 9, 40])
def test_chains_behind_long_contexts(hd, Hq, Hkv, n):
    c = case([n, 1, n], [3000, 1234, 15], Hq, Hkv, hd, seed=n)
    out, err = attend(c, max_len=n)
    assert not any(err)
    check(c, out, 0, 0)
    again, _ = attend(c, max_len=n)
    assert torch.equal(out, again)
    out, err = attend(c, window=700, sinks=20, max_len=n)
    check(c, out, 700, 20)


def test_a_prompt_in_parts_is_the_prompt():
    c = case([400], [0], 8, 2, 128, seed=3)
    want = oracle(c, 90, 5)
    out, _ = attend(c, 90, 5)
    check(c, out, 90, 5, want=want)
    for first, n in ((0, 1), (1, 255), (256, 144)):
        part = dict(c, q=c["q"][first:first + n], cu=whole([0, n]), prefix=whole([first]), lens=[n])
        got, err = attend(part, 90, 5)
        assert err == [0]
        check(c, got, 90, 5, want=[x[first:first + n] for x in want])


def test_step_equals_a_prompt_of_one():
    c = case([1] * 5, [9, 400, 2000, 16, 31], 8, 2, 128, seed=4)
    a, _ = attend(c, 100, 4)
    b, _ = attend(dict(c, step=True), 100, 4)
    want = oracle(c, 100, 4)
    check(c, a, 100, 4, want=want)
    check(c, b, 100, 4, want=want)


def test_large_scores_and_scales():
    c = case([150], [60], 4, 2, 128, seed=5, scale=30.0)
    out, _ = attend(c)
    check(c, out, 0, 0)
    for scale in (0.0, -0.3, 1e-30):
        out, _ = attend(c, sm_scale=scale)
        check(c, out, 0, 0, scale=scale)


def test_padded_step_leaves_rows_alone():
    prefix = [100, -5, 3, 40]
    c = case([1, 0, 1, 0], [100, 0, 3, 0], 4, 2, 128, seed=6)
    # a padded batch: rows 1 and 3 hold no sequence, and their numbers are whatever they are
    q = torch.full((4, 4, 128), float("nan"), dtype=BF, device=DEV)
    q[0], q[2] = c["q"][0], c["q"][1]
    table = c["table"].clone()
    table[1], table[3] = -9, 1 << 30
    d = dict(c, q=q, table=table, prefix=whole(prefix), lens=[1] * 4, step=True)
    out, err = attend(d, live=whole([1, 0, 1, 0]))
    assert err == [0] * 4 and (out[1] == 7).all() and (out[3] == 7).all()
    check(c, out[[0, 2]], 0, 0)


def test_rows_of_no_sequence_are_left_alone():
    c = case([20, 30], [5, 0], 4, 2, 64, seed=7)
    q = torch.full((90, 4, 64), float("nan"), dtype=BF, device=DEV)
    q[13:63] = c["q"]
    out, err = attend(dict(c, q=q, cu=whole([13, 33, 63])), max_len=90)
    assert err == [0, 0] and (out[:13] == 7).all() and (out[63:] == 7).all()
    check(c, out[13:63], 0, 0)
    none = dict(c, q=q[:0], cu=whole([0, 0, 0]))
    out, err = attend(none)
    assert err == [0, 0] and out.shape[0] == 0


def test_output_rows_may_lie_apart():
    c = case([33], [12], 4, 2, 128, seed=8)
    big = torch.full((33, 4 * 128 + 96), 5.0, dtype=BF, device=DEV)
    out = big[:, 32:32 + 512].unflatten(1, (4, 128))
    attend(c, out=out)
    check(c, out, 0, 0)
    assert (big[:, :32] == 5).all() and (big[:, 544:] == 5).all()


@pytest.mark.parametrize("step", [False, True])
def test_bad_sequences_are_reported_and_left_unwritten(step):
    c = case([1] * 6, [100, 20, 30, 900, 60, 900], 4, 2, 128, seed=9, step=step)
    table, prefix = c["table"].clone(), c["prefix"].clone()
    table[0, 3] = -1                    # a hole that a query sees
    table[1, 1] = c["k"].shape[0]       # past the cache
    prefix[2] = -1
    prefix[3] = table.shape[1] * 16     # no slot for the token
    prefix[4] = 2 ** 31 - 1
    out, err = attend(dict(c, table=table, prefix=prefix))
    assert err == [tv.TV_ERR_BAD_BLOCK] * 2 + [tv.TV_ERR_CAPACITY] * 3 + [0]
    assert (out[:5] == 7).all()
    check(c, out, 0, 0, rows=[5])
    # behind a window the hole is not seen
    out, err = attend(dict(c, table=table, prefix=prefix), window=30)
    assert err == [0, tv.TV_ERR_BAD_BLOCK] + [tv.TV_ERR_CAPACITY] * 3 + [0]
    check(c, out, 30, 0, rows=[0, 5])


@pytest.mark.parametrize("cu", [[0, 20, 10], [0, 20, 99], [-1, 20, 30], [5, 0, 30], [0, 25, 30]])
def test_bad_lengths_are_reported(cu):
    c = case([20, 10], [0, 0], 4, 2, 64, seed=10)
    out, err = attend(dict(c, cu=whole(cu)), max_len=20)
    assert err == [tv.TV_ERR_BAD_SEQLEN] * 2 and (out == 7).all()


def test_small_workspace_is_refused():
    c = case([1], [40000], 2, 1, 128, seed=11, step=True)
    need = tv.tv_window_attn_workspace_size(1, 1, 1, 2, 1, 128, c["table"].shape[1])
    if need:
        with pytest.raises(tv.TVError):
            attend(c, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    out, err = attend(c, workspace=torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV))
    assert err == [0]
    check(c, out, 0, 0)


@pytest.mark.parametrize("lens,prefix,step", [([60, 5], [7, 300], False), ([1, 1], [900, 4000], True), ([4, 4], [2000, 50], False)])
def test_graph_replays_and_other_streams(lens, prefix, step):
    c = case(lens, prefix, 8, 2, 128, seed=12, step=step)
    out, _ = attend(c, 500, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = attend(c, 500, 3, stream=side)
    assert torch.equal(out, got)
    again = torch.full_like(out, 7.0)
    err = torch.full((2,), 9, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if step:
            tv.tv_window_attn_step(c["q"], c["k"], c["v"], c["table"], c["prefix"], again, err, window=500, sinks=3)
        else:
            tv.tv_window_attn_prompt(c["q"], c["k"], c["v"], c["table"], c["cu"], c["prefix"], again, err, window=500, sinks=3)
    for shift in (0, 7):  # the same graph after the sequences moved on
        prefix_now = [p - shift for p in prefix]
        c["prefix"].copy_(whole(prefix_now))
        graph.replay()
        torch.cuda.synchronize()
        assert err.tolist() == [0, 0]
        check(dict(c, before=prefix_now), again, 500, 3)
        c["prefix"].copy_(whole(prefix))


@pytest.mark.parametrize("step", [False, True])
def test_offsets_past_32_bits(step):
    # 2^19 + some pages of 8 heads: elements past 2^33 of either cache
    blocks, Hkv, hd = (1 << 19) + 64, 8, 128
    c = case([1] if step else [70], [500], 16, Hkv, hd, seed=13, step=step, poison=False)
    big = [torch.empty(blocks, Hkv, 16, hd, dtype=BF, device=DEV) for _ in range(2)]
    used = c["k"].shape[0]
    for dst, src in zip(big, (c["k"], c["v"])):
        dst[-used:] = src
    moved = dict(c, k=big[0], v=big[1], table=torch.where(c["table"] < used, c["table"] + blocks - used, c["table"]))
    out, err = attend(moved, 300, 2)
    assert err == [0]
    check(c, out, 300, 2)
    del big, moved
    torch.cuda.empty_cache()


def test_sequences_do_not_touch_each_other():
    c = case([90, 80], [30, 40], 4, 2, 128, seed=14)
    out, _ = attend(c)
    one = torch.tensor(c["real"][1][:8], device=DEV).long()
    k = c["k"].clone()
    k[one] = float("nan")
    got, err = attend(dict(c, k=k))
    assert err == [0, 0] and torch.equal(out[:90], got[:90])


def test_prompts_long_enough_for_many_tiles():
    c = case([1500, 700], [0, 900], 8, 2, 128, seed=15)
    for window, sinks in ((0, 0), (256, 130)):
        out, err = attend(c, window, sinks)
        assert not any(err)
        rows = np.r_[0:3, 250:260, 1020:1030, 1490:1510, 2190:2200]
        # the oracle on those rows alone: each a sequence of one token
        starts, before = list(range(len(rows))), [int(r) if r < 1500 else int(r) - 1500 + 900 for r in rows]
        part = dict(c, q=c["q"][torch.tensor(rows, device=DEV)], starts=starts, lens=[1] * len(rows), before=before,
                    real=c["real"][[0 if r < 1500 else 1 for r in rows]])
        check(part, out[torch.tensor(rows, device=DEV)], window, sinks)
    assert np.isfinite(f64(out)).all()


@pytest.mark.parametrize("hd,Hq", [(64, 8), (128, 8), (256, 8)])
def test_units_of_one_and_two_row_tiles_side_by_side(hd, Hq):
    # a CTA's run holds sequences of few query rows behind many keys, then ones of many rows, in any order
    rng = np.random.default_rng(hd)
    lens = [int(x) for x in rng.choice([3, 20, 33, 64, 70], size=150)]
    prefix = [int(x) for x in rng.integers(300, 900, size=150)]
    c = case(lens, prefix, Hq, 2, hd, seed=16)
    for window, sinks in ((0, 0), (400, 4)):
        out, err = attend(c, window, sinks, max_len=70)
        assert not any(err)
        rows = np.sort(rng.choice(sum(lens), size=120, replace=False))
        seq = np.searchsorted(np.cumsum(lens), rows, side="right")
        before = [prefix[b] + int(r) - c["starts"][b] for b, r in zip(seq, rows)]
        at = torch.tensor(rows, device=DEV)
        part = dict(c, q=c["q"][at], starts=list(range(len(rows))), lens=[1] * len(rows), before=before, real=c["real"][seq])
        check(part, out[at], window, sinks)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("shape", ["rising", "jumps", "falling"])
@pytest.mark.parametrize("lens,prefix,Hq,step", [([300, 20], [100, 400], 4, False), ([2, 90], [700, 333], 8, False),
                                                 ([1, 1, 1], [50, 500, 1000], 4, True)])
def test_scores_that_outgrow_the_maximum_held(hd, shape, lens, prefix, Hq, step):
    # scores that climb by more than fp32 could hold against an early maximum, by steps inside and between tiles
    c = case(lens, prefix, Hq, 2, hd, seed=17, scale=0.1, step=step, poison=False)
    u = torch.randn(hd, generator=torch.Generator().manual_seed(1)).sign()
    c["q"] = (c["q"].float().cpu() + u).to(BF).to(DEV)
    jumps = np.array([70, 100, 129, 200, 333, 600])
    for b, (p, n) in enumerate(zip(prefix, lens)):
        at = np.arange(p + n)
        size = {"rising": at * 1.0, "falling": 1000.0 - at, "jumps": 40.0 * np.searchsorted(jumps, at)}[shape]
        block, row = torch.tensor(c["real"][b][at // 16], device=DEV).long(), torch.tensor(at % 16, device=DEV).long()
        k = 0.05 * torch.randn(len(at), 2, hd, generator=torch.Generator().manual_seed(b))
        k += torch.tensor(size, dtype=torch.float32)[:, None, None] * hd ** -0.5 * u
        c["k"][block, :, row] = k.to(BF).to(DEV)
    for window, sinks in ((0, 0), (150, 70)):
        out, err = attend(c, window, sinks)
        assert not any(err)
        check(c, out, window, sinks)


@pytest.mark.parametrize("step", [True, False])
def test_more_sequences_than_threads(step):
    rng = np.random.default_rng(18)
    B = 500
    lens = [1] * B if step else [int(x) for x in rng.choice([0, 1, 3, 5], size=B)]
    prefix = [int(x) for x in rng.integers(0, 200, size=B)]
    live = rng.random(B) < 0.8
    c = case(lens, prefix, 16, 2, 64, seed=18, step=step)
    out, err = attend(c, 90, 2, live=whole(live) if step else None, max_len=max(lens))
    assert not any(err)
    want = oracle(c, 90, 2)
    rows = np.nonzero(live)[0] if step else np.arange(sum(lens))
    check(c, out, 90, 2, rows=rows, want=want)
    if step:
        assert (out[torch.tensor(~live, device=DEV)] == 7).all()


def test_two_calls_on_two_streams_at_once():
    cases = [case([200, 40], [60, 300], 8, 2, 128, seed=19), case([1] * 4, [900, 20, 1500, 333], 8, 2, 128, seed=20, step=True)]
    want = [attend(c, 400, 3)[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.full_like(w, 7.0) for w in want]
    errs = [torch.full((len(c["lens"]),), 9, dtype=torch.int32, device=DEV) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, out, err in zip(cases, streams, outs, errs):
            if c["step"]:
                tv.tv_window_attn_step(c["q"], c["k"], c["v"], c["table"], c["prefix"], out, err, window=400, sinks=3, stream=s)
            else:
                tv.tv_window_attn_prompt(c["q"], c["k"], c["v"], c["table"], c["cu"], c["prefix"], out, err, window=400, sinks=3,
                                         stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and not any(e.any() for e in errs)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 1)])
@pytest.mark.parametrize("climb", [False, True])
def test_units_cut_among_several_ctas(hd, Hq, Hkv, climb):
    # units of so many keys that their parts meet in the workspace: whole ones, one row tile, ragged ends; and scores that
    # climb, so that a part's maximum tells nothing about the next one's
    lens, prefix = [130, 5, 64, 2], [4100, 2900, 1800, 40]
    c = case(lens, prefix, Hq, Hkv, hd, seed=19, scale=0.1 if climb else 1.5, poison=not climb)
    if climb:
        u = torch.randn(hd, generator=torch.Generator().manual_seed(2)).sign()
        c["q"] = (c["q"].float().cpu() + u).to(BF).to(DEV)
        for b, (p, n) in enumerate(zip(prefix, lens)):
            at = np.arange(p + n)
            block, row = torch.tensor(c["real"][b][at // 16], device=DEV).long(), torch.tensor(at % 16, device=DEV).long()
            k = 0.05 * torch.randn(len(at), Hkv, hd, generator=torch.Generator().manual_seed(b))
            k += torch.tensor(30.0 * (at // 333), dtype=torch.float32)[:, None, None] * hd ** -0.5 * u
            c["k"][block, :, row] = k.to(BF).to(DEV)
    for window, sinks in ((0, 0), (2500, 40)):
        out, err = attend(c, window, sinks)
        assert not any(err)
        check(c, out, window, sinks)
        again, _ = attend(c, window, sinks)
        assert torch.equal(out, again)
