"""Pins of the oracle's new-token definitions (positions, norm, rotation,
windowed attention) against plain loops and closed values, on the CPU."""
import math

import numpy as np
import pytest

import oracle


def table(rows, base=10000.0):
    a = np.arange(rows)[:, None] * base ** (-np.arange(32) / 32)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


def test_positions_by_hand():
    assert oracle.token_positions([5, 2, 0], None, 3).tolist() == [[2, 3, 4], [-1, 0, 1], [-1, -1, -1]]
    assert oracle.token_positions([5, 2, 7], [1, 3, 0], 3).tolist() == [[4, -1, -1], [-1, 0, 1], [-1, -1, -1]]


def test_norm_by_hand():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(oracle.rms_norm(x, None, 1e-300), x / math.sqrt(12.5), rtol=1e-15)
    assert np.allclose(oracle.rms_norm(x, np.array([2.0, -1.0]), 1.5), [[6 / math.sqrt(14.0), -4 / math.sqrt(14.0)]])
    assert oracle.rms_norm(x, None, 0.0) is x


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_is_a_complex_product_and_relative(halves):
    g = np.random.default_rng(1)
    tab = table(50)
    q, k = g.standard_normal(64), g.standard_normal(64)
    for i in range(32):
        ia, ib = (i, i + 32) if halves else (2 * i, 2 * i + 1)
        z = complex(q[ia], q[ib]) * complex(tab[7, i], tab[7, 32 + i])
        r = oracle.rotate(q, tab[7], halves)
        assert abs(complex(r[ia], r[ib]) - z) < 1e-12
    dots = [oracle.rotate(q, tab[a], halves) @ oracle.rotate(k, tab[a - 5], halves) for a in (5, 20, 49)]
    assert np.allclose(dots, dots[0], atol=1e-10)  # only the distance counts


def test_window_keys_by_loops():
    for p in (0, 1, 5, 40):
        for w in (1, 3, 41, 100):
            for k in (0, 1, 4, 60):
                want = [t for t in range(p + 1) if p - t < w or t < k]
                assert oracle.window_keys(p, w, k).tolist() == want


def test_window_decode_against_dense_and_by_brute_force():
    g = np.random.default_rng(2)
    kv = g.standard_normal((8, 64, 576))
    bt = np.array([[3, 1, 6], [0, 7, 2]])
    q = g.standard_normal((2, 2, 3, 576))
    lens = [150, 9]
    sc = 0.07
    o, l = oracle.window_decode(q, kv, bt, lens, None, sc, 10 ** 6, 0)
    do, dl = oracle.dense_decode(q, kv, bt, np.array(lens), sc, True)
    assert np.allclose(o, do) and np.allclose(l, dl)
    sink = np.array([0.3, -1.0, 2.0])
    o, l = oracle.window_decode(q, kv, bt, lens, [1, 2], sc, 5, 2, sink)
    for b, j, pos in ((0, 0, 149), (1, 0, 7), (1, 1, 8)):
        for h in range(3):
            num, den = np.zeros(512), 0.0
            for t in range(pos + 1):
                if pos - t < 5 or t < 2:
                    key = kv[bt[b, t // 64], t % 64]
                    e = math.exp(sc * float(q[b, j, h] @ key))
                    num += e * key[:512]
                    den += e
            assert math.isclose(l[b, h, j], math.log(den), rel_tol=1e-12)
            assert np.allclose(o[b, j, h], num / (den + math.exp(sink[h])))
    assert np.all(o[0, 1] == 0) and np.all(np.isneginf(l[0, :, 1]))  # padding
