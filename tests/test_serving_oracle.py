"""Pins of the serving oracle by hand-worked numbers (CPU)."""

import numpy as np

from oracle import serving_oracle as S


def test_e4m3_table():
    assert S.E4M3.size == 127 and S.E4M3[0] == 0 and S.E4M3[1] == 2.0 ** -9 and S.E4M3[-1] == 448
    assert S.E4M3[0x38] == 1.0 and np.all(np.diff(S.E4M3) > 0)


def test_codes_by_hand():
    x = np.zeros((1, 128))
    # group 0: amax 6 gives scale 1; borders go to the even code
    x[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, 0.74, 1.3, 2.6, 5.1, -5, 0]
    # group 1: amax 7: 7/6 = 1.1667 between 1.125 and 1.25, nearer 1.125; 7/1.125 = 6.22 stays 6
    x[0, 16] = 7
    code, bits = S.quantise(x)
    assert bits[0, 0] == 0x38 and S.E4M3[bits[0, 1]] == 1.125 and not bits[0, 2:].any()
    assert code[0, :16].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 9, 1, 3, 5, 7, 14, 0]
    v = S.values(code, bits)
    assert v[0, 16] == 6.75 and v[0, 1] == -6 and v[0, 8] == 4 and v[0, 14] == -4
    # the largest scale saturates, a power of two moves the range exactly
    assert S.round_trip(np.full((1, 128), 1e4))[0, 0] == 448 * 6
    assert np.array_equal(S.round_trip(x * 2.0 ** -20, 2.0 ** -20), v * 2.0 ** -20)
    assert np.isnan(S.round_trip(np.where(np.arange(128) == 3, np.inf, 1.0)[None])[0, :16]).all()


def test_window_and_sinks_by_hand():
    see = S.visible([0, 3, 5], np.arange(6), 2, 1)
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 0, 1, 1]]
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((n, 128)) for n in (3, 6, 6))
    o, lse, _, _ = S.attend(q, k, v, see, 0.1)
    assert np.allclose(o[0], v[0])
    w = np.exp(0.1 * q[2] @ k[[0, 4, 5]].T)
    assert np.allclose(o[2], w @ v[[0, 4, 5]] / w.sum()) and np.isclose(lse[2], np.log(w.sum()))
    o, lse, _, _ = S.attend(q, k, v, np.zeros((3, 6), bool), 0.1)
    assert not o.any() and np.isneginf(lse).all()


def test_norm_rotation_by_hand():
    x = np.zeros((1, 1, 1, 128))
    x[..., 0], x[..., 64] = 3.0, 4.0
    y, _ = S.qk_norm_rope(x, None, [[1]], 10000.0, 0.0)
    n = np.sqrt(128) / 5  # 1 / sqrt(25 / 128)
    assert np.allclose(y[0, 0, 0, [0, 64]], [n * (3 * np.cos(1) - 4 * np.sin(1)), n * (3 * np.sin(1) + 4 * np.cos(1))])


def test_extend_by_hand():
    table = np.array([[7, -1, -1], [-1, -1, -1]])
    t, slots, pos, head = S.extend(table, [15, 0], [18, 2], [9, 8, 7, 5, 3], 3, 4, 16)
    assert t.tolist() == [[7, 5, -1], [3, -1, -1]] and head == 5
    assert slots.tolist() == [[7 * 16 + 15, 80, 81, -1], [48, 49, -1, -1]]
    assert pos.tolist() == [[15, 16, 17, -1], [0, 1, -1, -1]]
