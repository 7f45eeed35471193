"""What pins the float64 oracle of the mixers: hand-worked cases, closed forms, and identities."""
import numpy as np

from oracle import mixers


def test_plan_by_hand():
    table = np.array([[7, -1, -1], [4, 5, -1], [-1, -1, -1]])
    t, slots, rows, total, used = mixers.cache_plan([16, 20, 0], [1, 3, 17], 16, [9, 2, 6, 8], table, 23)
    assert t.tolist() == [[7, 9, -1], [4, 5, -1], [2, 6, -1]]
    assert slots.tolist() == [9 * 16] + [5 * 16 + 4, 5 * 16 + 5, 5 * 16 + 6] + list(range(32, 48)) + [96, -1, -1]
    assert rows.tolist() == [0, 1, 4, 21] and total.tolist() == [17, 23, 17] and used == 3


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    o, _ = mixers.prompt_attention(q, k, v, [0, 5], [0, 5], 0.3)
    assert np.allclose(o[0], v[0])  # one key: its value
    o, _ = mixers.prompt_attention(0 * q, k, v, [0, 5], [0, 5], 0.3)
    assert np.allclose(o[4, 0], v[:, 0].mean(0))  # equal scores: the mean
    o, _ = mixers.prompt_attention(q[:3], k[:1], v[:1], [0, 3], [0, 1], 0.3)
    assert (o[:2] == 0).all() and np.allclose(o[2], v[0])
    two = np.array([[0.0], [np.log(3.0)]])
    o, _ = mixers.prompt_attention(np.ones((1, 1, 1)), two[:, None], np.array([1.0, 5.0])[:, None, None], [0, 1], [0, 2], 1.0)
    assert np.isclose(o[0, 0, 0], (1 + 3 * 5) / 4)


def test_a_chain_of_drafts_is_a_prompts_last_rows():
    rng = np.random.default_rng(1)
    L, n = 23, 4
    q, k, v = rng.standard_normal((n, 2, 8)), rng.standard_normal((L, 1, 8)), rng.standard_normal((L, 1, 8))
    kc, vc = np.zeros((4, 1, 16, 8)), np.zeros((4, 1, 16, 8))
    kc, vc = mixers.cache_write(k, v, [2 * 16 + i for i in range(16)] + [i for i in range(7)], kc, vc)
    a, _ = mixers.prompt_attention(q, k, v, [0, n], [0, L], 0.4)
    for words in (None, [1, 3, 7, 15]):
        b, _ = mixers.tree_attention(q, kc, vc, [[2, 0]], [L], [0, n], words, 0.4)
        assert np.allclose(a, b)
    b, _ = mixers.tree_attention(q, kc, vc, [[2, 0]], [L], [0, n], [1, 2, 0b101, 0b1010], 0.4)
    assert np.allclose(a[0], b[0]) and not np.allclose(a[1], b[1])


def test_delta_closed_forms():
    rng = np.random.default_rng(2)
    D = 6
    k = np.eye(D)[:, None]  # orthonormal keys, full steps, no decay: the state maps each key to its value
    v = rng.standard_normal((D, 1, D))
    one, zero = np.ones((D, 1)), np.zeros((D, 1))
    o, S, _ = mixers.gated_delta(k, k, v, zero, one, [0, D], np.zeros((1, 1, D, D)), False, 1.0)
    assert np.allclose(S[0, 0], v[:, 0]) and np.allclose(o, v)
    k = np.repeat(k[:1], 2, 0)  # the same key again: its value is replaced
    _, S, _ = mixers.gated_delta(k, k, v[:2], zero[:2], one[:2], [0, 2], np.zeros((1, 1, D, D)), False, 1.0)
    assert np.allclose(S[0, 0, 0], v[1, 0]) and (S[0, 0, 1:] == 0).all()
    half = np.full((1, 1), np.log(0.5))
    _, S, _ = mixers.gated_delta(k[:1], k[:1], v[:1], half, 0 * half, [0, 1], np.ones((1, 1, D, D)), False, 1.0)
    assert np.allclose(S, 0.5)  # no step: only the decay


def test_delta_step_is_the_gradient_of_half_the_squared_error():
    """S - e^g S = -beta dE/dS at e^g S, E = |v - S^T k|^2 / 2, by central differences."""
    rng = np.random.default_rng(3)
    D = 5
    S0, k, v = rng.standard_normal((1, 1, D, D)), rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))
    g, beta = np.full((1, 1), -0.3), np.full((1, 1), 0.7)
    _, S, _ = mixers.gated_delta(k, k, v, g, beta, [0, 1], S0, False, 1.0)
    base = np.exp(-0.3) * S0[0, 0]
    err = lambda M: 0.5 * np.sum((v[0, 0] - M.T @ k[0, 0]) ** 2)  # noqa: E731
    for i in range(D):
        for j in range(D):
            d = np.zeros((D, D))
            d[i, j] = 1e-5
            grad = (err(base + d) - err(base - d)) / 2e-5
            assert np.isclose(S[0, 0, i, j], base[i, j] - 0.7 * grad, atol=1e-8)


def test_delta_splits_anywhere():
    rng = np.random.default_rng(4)
    T, D = 11, 4
    q, k, v = (rng.standard_normal((T, 2, D)) for _ in range(3))
    g, beta = -rng.random((T, 2)), rng.random((T, 2))
    S0 = rng.standard_normal((1, 2, D, D))
    o, S, _ = mixers.gated_delta(q, k, v, g, beta, [0, T], S0, True, 0.5)
    for c in (1, 6):
        o1, S1, _ = mixers.gated_delta(q[:c], k[:c], v[:c], g[:c], beta[:c], [0, c], S0, True, 0.5)
        o2, S2, _ = mixers.gated_delta(q[c:], k[c:], v[c:], g[c:], beta[c:], [0, T - c], S1, True, 0.5)
        assert np.allclose(np.concatenate([o1, o2]), o) and np.allclose(S2, S)
