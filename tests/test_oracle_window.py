"""Pins of the windowed attention's oracle: closed forms, and the distribution that acceptance has to leave alone."""
import itertools

import numpy as np
import pytest

from oracle import window as O


def test_rotation_keeps_lengths_and_turns_by_the_difference_of_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 64))
    for rotary in (0, 16, 32, 64):
        a, b = O.rotate(q, 1000, rotary, 1e4), O.rotate(k, 990, rotary, 1e4)
        c, d = O.rotate(q, 17, rotary, 1e4), O.rotate(k, 7, rotary, 1e4)
        assert np.isclose(np.linalg.norm(a), np.linalg.norm(q)) and np.isclose(a @ b, c @ d)
        assert np.array_equal(a[rotary:], q[rotary:])
    assert np.allclose(O.rotate(np.eye(2)[0], 0.5, 2, 1e4), [np.cos(0.5), np.sin(0.5)])


def test_norm_then_rotation():
    x = np.full((1, 1, 64), 3.0)
    y = O.norm_rotate(x, np.full(64, 2.0), [0], 64, 1e4, 0.0)
    assert np.allclose(y, 2.0)
    assert np.allclose(O.norm_rotate(x, np.full(64, 2.0), [0], 64, 1e4, 0.0, weight_offset=1.0), 3.0)
    assert np.array_equal(O.norm_rotate(x, None, [5], 0, 1e4, 0.0, norm=False), x)


def test_visible_positions():
    assert O.visible(5, 0, 0).tolist() == [0, 1, 2, 3, 4, 5] == O.visible(5, 99, 0).tolist()
    assert O.visible(5, 2, 0).tolist() == [4, 5] and O.visible(5, 1, 2).tolist() == [0, 1, 5]
    assert O.visible(2, 1, 9).tolist() == [0, 1, 2] and O.visible(0, 1, 0).tolist() == [0]


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 3, 1, 16, 4))
    table = np.array([[2, 0]])
    q = rng.standard_normal((5, 2, 4))
    at = lambda c, j: c[table[0, j // 16], 0, j % 16]  # noqa: E731
    o = O.window_attn(q, k, v, table, [0], [5], [14], 1, 0, 0.5)[0]      # each token sees itself alone
    assert np.allclose(o, np.stack([[at(v, 14 + i)] * 2 for i in range(5)]))
    o, size, reach = O.window_attn(np.zeros((5, 2, 4)), k, v, table, [0], [5], [14], 3, 2, 0.5)   # equal weights
    seen = [0, 1, 16, 17, 18]
    assert np.allclose(o[4], np.mean([at(v, j) for j in seen], axis=0))
    assert np.allclose(size[4], np.mean([np.abs(at(v, j)) for j in seen], axis=0)) and not reach.any()


def spread(parents, p, q, steps, draws):
    """Probability of each continuation (tokens after node 0, three of them by p) over a grid of random numbers, the
    drafted tokens drawn from q."""
    N, V = p.shape
    got = {}
    grid = (np.arange(steps) + 0.5) / steps
    for tokens in draws:
        weight = np.prod([q[parents[i], tokens[i]] if q is not None else 1.0 for i in range(1, N)])
        for u in itertools.product(grid, repeat=N):
            path, after = O.accept_sample(parents, tokens, p, q, u, N)
            out = tuple(tokens[i] for i in path[1:]) + (after,)
            got[out] = got.get(out, 0.0) + weight / steps ** N
    return got


@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("parents", [[-1, 0], [-1, 0, 0]])
def test_the_first_token_is_distributed_as_the_target(parents, known):
    # a number from the middles of n equal parts lies on a side of a border with a probability that is off by 1/(2 n) at
    # most: each test has one border, the draw of a token two
    p = np.tile(np.array([10, 6, 3, 1]) / 20, (len(parents), 1))
    q = np.tile(np.array([4, 4, 2, 10]) / 20, (len(parents), 1)) if known else None
    kids = len(parents) - 1
    draws = [(0,) + d for d in itertools.product(range(4), repeat=kids)] if known else [(0, 2, 1)[:1 + kids]]
    n = 60 if kids == 1 else 24
    got = spread(parents, p, q, n, draws)
    first = np.zeros(4)
    for out, w in got.items():
        first[out[0]] += w
    assert np.allclose(first, p[0], rtol=0, atol=(kids / 2 + 1) / n), first


def test_acceptance_corner_cases():
    p = np.array([[0.5, 0.5, 0.0], [0.0, 0.0, 1.0]])
    assert O.accept_sample([-1, 0], [0, 1], p, None, [0.0, 0.49], 2) == ([0, 1], 2)
    assert O.accept_sample([-1, 0], [0, 1], p, None, [0.0, 0.5], 2) == ([0], 0)       # refused, and left out of the draw
    assert O.accept_sample([-1, 0], [0, 1], p, None, [0.0, 0.49], 1) == ([0], 0)      # no room for a second node
    assert O.accept_sample([-1, 0], [0, 7], p, None, [0.6, 0.0], 2) == ([0], 1)       # no such token
    assert O.accept_sample([-1, 0], [0, 0], p, p, [0.6, 0.999], 2) == ([0, 1], 2)     # p = q: never refused
    assert O.accept_sample([-1, 0], [0, 0], np.zeros((2, 3)), p, [0.6, 0.0], 2) is None
