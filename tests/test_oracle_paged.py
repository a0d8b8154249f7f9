"""Pins of the paged-cache oracle: brute force, closed forms, the plain attention oracle."""
import math

import numpy as np
import pytest

from oracle import attention, paged


def _normal(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("n_kv,n_q,causal", [(1, 1, True), (5, 1, True), (5, 5, True), (7, 3, True), (7, 3, False),
                                             (2, 4, True), (0, 2, True), (0, 2, False)])
def test_attend_by_scalar_brute_force(n_kv, n_q, causal):
    q, k, v = _normal(1, n_q, 4, 3), _normal(2, n_kv, 2, 3), _normal(3, n_kv, 2, 3)
    out, lse, weight, reach = paged.attend(q, k, v, causal)
    want_w = np.zeros((2, n_kv))
    for i in range(n_q):
        for h in range(4):
            g = h // 2
            keys = [j for j in range(n_kv) if not causal or j <= n_kv - n_q + i]
            e = {j: math.exp(sum(q[i, h, c] * k[j, g, c] for c in range(3)) / math.sqrt(3)) for j in keys}
            total = sum(e.values())
            for c in range(3):
                want = sum(e[j] / total * v[j, g, c] for j in keys) if keys else 0.0
                assert abs(out[i, h, c] - want) < 1e-13
                size = sum(e[j] / total * abs(v[j, g, c]) for j in keys) if keys else 0.0
                assert abs(reach[i, h, c] - size) < 1e-13
            assert lse[i, h] == pytest.approx(math.log(total), abs=1e-13) if keys else lse[i, h] == -math.inf
            for j in keys:
                want_w[g, j] += e[j] / total
    assert np.allclose(weight, want_w, atol=1e-13)


def test_attend_without_a_mask_is_the_chunk_attention_oracle():
    q, k, v = _normal(4, 6, 3, 8), _normal(5, 11, 3, 8), _normal(6, 11, 3, 8)
    assert np.allclose(paged.attend(q, k, v, False)[0], attention.attend(q, k, v), atol=1e-13)


def test_weights_add_up_to_the_rows_and_restart_for_the_chunk():
    q, k, v = _normal(7, 3, 4, 8), _normal(8, 9, 2, 8), _normal(9, 9, 2, 8)
    got = paged.attend(q, k, v, True)[2]
    assert np.allclose(got.sum(1), 3 * 2)
    assert got[0, -1] > 0 and (got[:, 6:] > 0).all()
    new = paged.accumulate(np.full((2, 9), 5.0), got, 3)
    assert np.allclose(new[:, :6], 5.0 + got[:, :6]) and np.allclose(new[:, 6:], got[:, 6:])
    assert np.array_equal(paged.accumulate(np.ones((2, 9)), np.zeros((2, 9)), 0), np.ones((2, 9)))


def test_kept_by_hand():
    w = np.array([0.0, 9.0, 1.0, 3.0, 3.0, np.nan, 2.0, 0.5])
    assert paged.kept(w, 8, 1, 1) == list(range(8))
    assert paged.kept(w, 4, 1, 1) == [0, 1, 3, 7]          # 9, then the earlier 3
    assert paged.kept(w, 5, 1, 1) == [0, 1, 3, 4, 7]
    assert paged.kept(w, 7, 1, 1) == [0, 1, 2, 3, 4, 6, 7]  # the NaN goes first
    assert paged.kept(w, 3, 3, 0) == [0, 1, 2]
    assert paged.kept(w, 3, 0, 3) == [5, 6, 7]
    assert paged.kept(np.array([0.0, -0.0, 0.0]), 2, 0, 0) == [0, 1]
    assert paged.kept(np.array([-1.0, np.inf, -np.inf]), 2, 0, 0) == [0, 1]
