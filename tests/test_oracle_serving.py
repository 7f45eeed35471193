"""What pins the float64 oracle of the operators around the linears: hand-worked cases and identities."""
import math

import numpy as np

from oracle import serving


def test_rotary_by_hand():
    x = np.array([1.0, 2, 3, 4, 5, 6])[None, None]
    f = np.array([math.pi / 2, math.pi])
    half, _ = serving.rotary(x, [1], f, 1.0, 4, pairs=False)  # (1, 3) by a quarter turn, (2, 4) by half a turn
    assert np.allclose(half[0, 0], [-3, -2, 1, -4, 5, 6])
    pairs, size = serving.rotary(x, [1], f, 2.0, 4, pairs=True)
    assert np.allclose(pairs[0, 0], [-4, 2, -6, -8, 5, 6])
    assert np.allclose(size[0, 0], [6, 6, 14, 14, 0, 0])


def test_rotary_depends_on_distance_and_turns_back():
    rng = np.random.default_rng(0)
    f, amp = serving.rotary_freqs(16, 1e4)
    assert amp == 1 and np.allclose(f, [1e4 ** (-i / 8) for i in range(8)])
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    for pairs in (False, True):
        dots = []
        for p in (0, 1234, 10 ** 9):
            a, b = serving.rotary(q, [p + 7], f, 1.0, 16, pairs)[0], serving.rotary(k, [p], f, 1.0, 16, pairs)[0]
            dots.append((a * b).sum())
        assert np.allclose(dots, dots[0])
        y, _ = serving.rotary(q, [991], f, 1.0, 16, pairs)
        assert np.allclose(serving.rotary(y, [991], f, 1.0, 16, pairs, inverse=True)[0], q)
        assert np.allclose(serving.rotary(y, [-991], f, 1.0, 16, pairs)[0], q)


def test_angles_far_away():
    assert math.isclose(serving.angle(10 ** 9, 1.0), math.remainder(1e9, 2 * math.pi), abs_tol=1e-6)
    assert serving.angle(0, 3.0) == 0 and math.isclose(serving.angle(-1, 1.0), -1.0)


def test_scaled_frequencies():
    f, _ = serving.rotary_freqs(64, 1e4)
    assert np.allclose(serving.rotary_freqs(64, 1e4, "linear", 4.0)[0], f / 4)
    b = serving.rotary_freqs(64, 1e4, "base", 4.0)[0]
    assert np.isclose(b[0], f[0]) and np.isclose(b[-1], f[-1] / 4)  # the fastest as it was, the slowest as in "linear"
    p, amp = serving.rotary_freqs(64, 1e4, "parts", 8.0, original=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(p[turns > 40], f[turns > 40]) and np.allclose(p[turns < 0.7], f[turns < 0.7] / 8)
    assert np.isclose(amp, 1 + 0.1 * math.log(8)) and (np.diff(p) < 0).all()


def test_adapter_by_hand():
    a = np.array([[[1.0, 0], [0, 1]], [[1, 1], [5, 5]]])
    b = np.array([[[1.0, 2]], [[3, 7]]])
    x, y = np.array([[1.0, 2], [3, 4], [5, 6]]), np.array([[10.0], [20], [30]])
    out, S, H = serving.adapter_linear(x, a, b, [1.0, -0.5], [2, 1], [0, 1, 2, 3], [0, -1, 1], y)
    assert out.tolist() == [[15.0], [20.0], [30 - 0.5 * 3 * 11]]
    assert S[1, 0] == 0 and H[2, 0] == 16.5


def test_logits_by_hand():
    x = np.array([[2.0, -2, 1, 0, 4], [2, -2, 1, 0, 4]])
    out = serving.logits_adjust(x, [0, 2], [[0, 1, 1, 4, 4]], [4], [3], fresh=[2, 4], repetition=[2.0], presence=[0.5], frequency=[0.25],
                                biases=[[(3, 1.0), (3, 7.0), (9, 1.0)]], mask=np.array([[0b11101], [0b11111]], dtype=np.int32))
    # prompt 0 1 1, generated 4; the first row's path is token 2, the second's tokens 2 and 4
    assert out[0].tolist() == [1.0, -np.inf, 0.5 - 0.75, 7.0, 2.0 - 0.75]
    assert out[1].tolist() == [1.0, -4.0, 0.5 - 0.75, 7.0, 2.0 - 0.5 - 0.5]
    tree = serving.logits_adjust(x, [0, 2], [[0]], [0], fresh=[2, 4], tree=[1, 2], presence=[1.0])
    assert tree[0].tolist() == [2, -2, 0, 0, 4] and tree[1].tolist() == [2, -2, 1, 0, 3]
