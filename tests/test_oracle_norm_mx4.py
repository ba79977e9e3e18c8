"""Pins of the norm and 4-bit oracles: closed forms, finite differences, the
format's hand-derived vectors, and properties of the nearest value."""

import numpy as np
import pytest

from oracle import mx4_ref, norm_ref


def test_norm_closed_forms():
    # a constant row: rms = |c|, so y = sign(c) w (eps = 0)
    w = np.array([1.0, 2.0, -3.0, 0.5])
    y, s, rstd = norm_ref.forward(np.full((2, 4), [[-4.0], [0.25]]), w, 0.0)
    assert np.array_equal(y, np.stack([-w, w])) and np.array_equal(rstd, [0.25, 4.0])
    # residual that cancels: only eps is left under the root
    x = np.arange(8.0).reshape(2, 4)
    y, s, rstd = norm_ref.forward(x, w, 0.25, res=-x)
    assert not s.any() and not y.any() and np.array_equal(rstd, [2.0, 2.0])
    # (3, 4): mean square 12.5
    y, _, _ = norm_ref.forward([[3.0, 4.0]], [1.0, 1.0], 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]], rtol=1e-15)


@pytest.mark.parametrize("T,d,eps", [(1, 4, 1e-6), (5, 24, 1e-2), (3, 1, 1e-3)])
def test_norm_gradients_by_differences(T, d, eps):
    g = np.random.default_rng(T + d)
    x, res, dy, ds = (g.standard_normal((T, d)) for _ in range(4))
    w = g.standard_normal(d)

    def loss(x, res, w):
        y, s, _ = norm_ref.forward(x, w, eps, res)
        return np.sum(y * dy) + np.sum(s * ds)

    _, s, rstd = norm_ref.forward(x, w, eps, res)
    dx, dw = norm_ref.backward(dy, s, w, rstd, ds)
    h = 1e-6
    for i in np.ndindex(T, d):
        e = np.zeros((T, d))
        e[i] = h
        num = (loss(x + e, res, w) - loss(x - e, res, w)) / (2 * h)
        num_r = (loss(x, res + e, w) - loss(x, res - e, w)) / (2 * h)
        assert abs(num - dx[i]) <= 1e-6 * (1 + abs(dx[i])) and abs(num_r - dx[i]) <= 1e-6 * (1 + abs(dx[i]))
    for c in range(d):
        e = np.zeros(d)
        e[c] = h
        num = (loss(x, res, w + e) - loss(x, res, w - e)) / (2 * h)
        assert abs(num - dw[c]) <= 1e-6 * (1 + abs(dw[c]))


def test_e2m1_hand_vectors():
    a = np.zeros((5, 32))
    # amax 6: s = 0; every border goes to the even code
    a[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2, 0.3, -0.25, 0.0, -0.0, 4.9, 5.1]
    a[1, 0] = 7.9           # still s = 0, saturates at 6
    a[2, 0], a[2, 1] = 8.0, 1.0   # s = 1: 8 -> 4 * 2, 1 -> 0.5 * 2
    a[4, 3] = np.inf
    q, s = mx4_ref.quantize_rows(a)
    v = mx4_ref.dequantize_rows(q, s)
    assert list(s[:, 0]) == [127, 127, 128, 0, 255]
    assert list(v[0, :16]) == [6, -6, 0, 1, 1, 2, 2, 4, 4, 0, 0.5, 0, 0, 0, 4, 6]
    assert q[0, 13] == 8 and q[0, 12] == 0  # the sign of zero
    assert v[1, 0] == 6 and v[2, 0] == 8 and v[2, 1] == 1 and not v[3].any()
    assert np.isnan(v[4]).all() and not q[4].any()


def test_e2m1_is_the_nearest_value_and_packs():
    g = np.random.default_rng(0)
    a = g.standard_normal((16, 160)) * np.exp(g.uniform(-60, 60, (16, 1)))
    q, s = mx4_ref.quantize_rows(a)
    assert np.array_equal(mx4_ref.unpack(mx4_ref.pack(q)), q)
    e = np.ldexp(1.0, s.astype(int) - 127)
    x = a.reshape(16, 5, 32) / e[:, :, None]
    v = mx4_ref.dequantize_rows(q, s).reshape(16, 5, 32) / e[:, :, None]
    assert np.abs(x).max() < 8 and np.abs(x).max(axis=2).min() >= 4
    grid = np.concatenate([-mx4_ref.VALUES, mx4_ref.VALUES])
    best = np.abs(x[..., None] - grid).min(axis=-1)
    assert np.array_equal(np.abs(x - v), best)
    # stored order: block b of row r at byte (b // 4 * M + r) * 4 + b % 4
    c = mx4_ref.scales_to_chunks(s)
    assert c.size == 2 * 16 * 4
    for r in range(16):
        for b in range(8):
            assert c[(b // 4 * 16 + r) * 4 + b % 4] == (s[r, b] if b < 5 else 0)
