"""Pins of the oracle's prompt definitions against plain loops, closed values and the absorbed form, on the CPU."""
import math

import numpy as np
import pytest

import oracle


def loops(q, k, v, n, m, scale, causal):
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    for j in range(n):
        keys = [t for t in range(m) if not causal or t <= j + m - n]
        s = [scale * sum(a * b for a, b in zip(q[j], k[t])) for t in keys]
        if s:
            lse[j] = math.log(math.fsum(math.exp(x) for x in s))
            for x, t in zip(s, keys):
                out[j] += math.exp(x - lse[j]) * v[t]
    return out, lse


@pytest.mark.parametrize("causal", [True, False])
def test_packed_attention_by_loops(causal):
    g = np.random.default_rng(0)
    q_lens, k_lens = [3, 0, 4, 2], [3, 2, 9, 1]
    cu_q, cu_k = [1] + (1 + np.cumsum(q_lens)).tolist(), [0] + np.cumsum(k_lens).tolist()
    q, k, v, r = g.standard_normal((cu_q[-1] + 2, 4, 192)), g.standard_normal((15, 2, 128)), g.standard_normal((15, 2, 128)), g.standard_normal((15, 64))
    for rope in (r, g.standard_normal((15, 2, 64))):
        out, lse, size = oracle.packed_attention(q, k, v, cu_q, cu_k, 0.07, causal, rope)
        for i in range(4):
            a, c, e = cu_q[i], cu_k[i], cu_k[i + 1]
            for h in range(4):
                key = np.concatenate([k[c:e, h // 2], rope[c:e] if rope.ndim == 2 else rope[c:e, h // 2]], 1)
                o, l = loops(q[a:a + q_lens[i], h], key, v[c:e, h // 2], q_lens[i], k_lens[i], 0.07, causal)
                assert np.allclose(out[a:cu_q[i + 1], h], o, atol=1e-12) and np.allclose(lse[h, a:cu_q[i + 1]], l, atol=1e-12)
        assert np.all(np.isnan(out[0])) and np.all(np.isnan(lse[:, -2:]))
        live = slice(1, -2)
        assert np.all(np.abs(out[live]) <= size[live] + 1e-12)


def test_the_absorbed_form_is_the_same():
    """Keys and values projected up per head against queries projected down onto the latent rows."""
    g = np.random.default_rng(1)
    h, n, m = 3, 4, 11
    c, r = g.standard_normal((m, 512)), g.standard_normal((m, 64))
    wk, wv = g.standard_normal((h, 128, 512)) / 20, g.standard_normal((h, 128, 512)) / 20
    q = g.standard_normal((n, h, 192))
    k, v = np.einsum("hdc,mc->mhd", wk, c), np.einsum("hdc,mc->mhd", wv, c)
    out, lse, _ = oracle.packed_attention(q, k, v, [0, n], [0, m], 0.072, True, r)
    absorbed = np.concatenate([np.einsum("nhd,hdc->nhc", q[..., :128], wk), q[..., 128:]], -1)
    for j in range(n):
        o, l = oracle.attend(absorbed[j], np.concatenate([c, r], 1)[:m - n + j + 1], 0.072)
        assert np.allclose(np.einsum("hc,hdc->hd", o, wv), out[j], atol=1e-12) and np.allclose(l, lse[:, j], atol=1e-12)


def test_merged_pieces_are_the_whole():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((5, 2, 128)), g.standard_normal((30, 2, 128)), g.standard_normal((30, 2, 128))
    whole = oracle.packed_attention(q, k, v, [0, 5], [0, 30], 0.1, False)
    parts = [oracle.packed_attention(q, k[a:z], v[a:z], [0, 5], [0, z - a], 0.1, False) for a, z in ((0, 7), (7, 7), (7, 30))]
    out, lse = oracle.merge_states(np.stack([p[0] for p in parts]), np.stack([p[1] for p in parts]))
    assert np.allclose(out, whole[0], atol=1e-13) and np.allclose(lse, whole[1], atol=1e-13)
    out, lse = oracle.merge_states(np.full((2, 1, 1, 3), np.nan), np.full((2, 1, 1), -np.inf))
    assert np.all(out == 0) and np.all(np.isneginf(lse))
    out, lse = oracle.merge_states(np.array([1.0, 4.0]).reshape(2, 1, 1, 1), np.log([[[1.0]], [[2.0]]]))
    assert abs(out.item() - 3.0) < 1e-14 and abs(lse.item() - math.log(3)) < 1e-14


def test_gathered_rows_by_hand():
    rows = np.arange(3 * 64 * 2.0).reshape(3, 64, 2)
    got = oracle.gather_rows(rows, [[2, 0], [1, -1]], [0, 3, 4], [63, 5])
    assert got.tolist() == [rows[2, 63].tolist(), rows[0, 0].tolist(), rows[0, 1].tolist(), rows[1, 5].tolist()]
