"""Pins of the fp64 mixer oracle: closed forms of the decayed recurrence, its relation to the gated
delta rule's oracle, and the norms' defining properties."""
import numpy as np

from oracle import gdn as G
from oracle import mixer as M


def _inputs(T, Hk, H, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, Hk, dk)), r.standard_normal((T, Hk, dk)), r.standard_normal((T, H, dv)),
            r.uniform(0.2, 1.0, (T, H)))


def test_outputs_are_the_decayed_score_sums():
    q, k, v, a = _inputs(9, 1, 2, 4, 3)
    S0 = np.random.default_rng(1).standard_normal((1, 2, 3, 4))
    o, S = M.linear_attn(q, k, v, a, [0, 9], S0, q_scale=0.5)
    for h in range(2):
        for t in range(9):
            want = 0.5 * np.prod(a[:t + 1, h]) * S0[0, h] @ q[t, 0]
            for j in range(t + 1):
                want = want + 0.5 * np.prod(a[j + 1:t + 1, h]) * (q[t, 0] @ k[j, 0]) * v[j, h]
            np.testing.assert_allclose(o[t, h], want, atol=1e-12)
        np.testing.assert_allclose(S[0, h] @ q[8, 0] * 0.5, o[8, h], atol=1e-12)


def test_equals_the_gated_delta_rule_on_orthogonal_keys():
    # with orthonormal keys, beta = 1 and S_0 = 0 the delta correction S k is always zero
    _, _, v, a = _inputs(4, 1, 1, 4, 4, seed=3)
    k = np.eye(4)[:, None, :]
    q = np.random.default_rng(5).standard_normal((4, 1, 4))
    o, S = M.linear_attn(q, k, v, a, [0, 4])
    state = np.zeros((1, 4, 4))
    for t in range(4):
        state = G.gdn_step(state, k[t], v[t], a[t], [1.0])
        np.testing.assert_allclose(o[t], G.gdn_output(state, q[t]), atol=1e-12)
    np.testing.assert_allclose(S[0], state, atol=1e-12)


def test_prompts_are_independent_and_cut_anywhere():
    q, k, v, a = _inputs(11, 2, 2, 4, 4, seed=7)
    o, S = M.linear_attn(q, k, v, a, [0, 4, 4, 11])
    o1, S1 = M.linear_attn(q[4:], k[4:], v[4:], a[4:], [0, 7])
    np.testing.assert_array_equal(o[4:], o1)
    np.testing.assert_array_equal(S[2], S1[0])
    assert not S[1].any()                                   # an empty prompt keeps its (zero) state
    whole, end = M.linear_attn(q, k, v, a, [0, 11])
    first, mid = M.linear_attn(q[:5], k[:5], v[:5], a[:5], [0, 5])
    rest, last = M.linear_attn(q[5:], k[5:], v[5:], a[5:], [0, 6], mid)
    np.testing.assert_allclose(np.concatenate([first, rest]), whole, atol=1e-12)
    np.testing.assert_allclose(last, end, atol=1e-12)


def test_norms():
    r = np.random.default_rng(2)
    x, g, w = r.standard_normal((5, 3, 8)), r.standard_normal((5, 3, 8)), r.standard_normal(8)
    n = M.rmsnorm(x, 0.0)
    np.testing.assert_allclose(np.mean(n * n, -1), 1.0, atol=1e-12)          # unit mean square
    np.testing.assert_allclose(M.rmsnorm(7 * x, 0.0), n, atol=1e-12)         # scale-free
    np.testing.assert_allclose(M.rmsnorm(x, 0.0, w, 1.0), n * (1 + w), atol=1e-12)
    np.testing.assert_allclose(M.silu(g) + M.silu(-g), g * np.tanh(g / 2), atol=1e-12)
    np.testing.assert_allclose(M.gated_rmsnorm(x, g, w, 0.0), n * w * M.silu(g), atol=1e-12)
    np.testing.assert_allclose(M.gated_rmsnorm(x, g, w, 0.0, True), M.rmsnorm(x * M.silu(g), 0.0) * w, atol=1e-12)
    y, res = x[:, 0], x[:, 1]
    out, nxt = M.residual_rmsnorm(y, res, 0.0, scale=0.5)
    np.testing.assert_allclose(out, res + 0.5 * y, atol=1e-12)
    np.testing.assert_allclose(nxt, M.rmsnorm(out, 0.0), atol=1e-12)
    out, _ = M.residual_rmsnorm(y, res, 0.0, post_weight=w, gate=g[:, 0], scale=2.0)
    np.testing.assert_allclose(out, res + 2.0 * g[:, 0] * M.rmsnorm(y, 0.0) * w, atol=1e-12)
