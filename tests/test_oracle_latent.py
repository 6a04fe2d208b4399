"""The float64 oracle of the latent-attention operators against hand-computed
numbers, closed forms and brute force."""
import math

import numpy as np
import pytest

from oracle import latent_attention as la


def test_two_keys_by_hand():
    # logits 0 and 1 (natural base): weights 1 / (1 + e) and e / (1 + e)
    q, k = np.array([[1.0, 0.0]]), np.array([[0.0, 5.0], [1.0, 7.0]])
    v = np.array([[2.0], [-4.0]])
    out, lse, p, mag, spread = la.rows_over_keys(q, k, v, [2], 1.0)
    e = math.e
    assert np.allclose(p, [[1 / (1 + e), e / (1 + e)]])
    assert np.allclose(out, [[(2 - 4 * e) / (1 + e)]]) and np.allclose(mag, [[(2 + 4 * e) / (1 + e)]])
    assert np.allclose(lse, math.log2(1 + e)) and np.allclose(spread, math.log2(e))


def test_masks_and_empty_rows():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 4)), rng.standard_normal((6, 4)), rng.standard_normal((6, 2))
    out, lse, p, _, _ = la.rows_over_keys(q, k, v, [0, 1, 6], 0.5)
    assert np.all(out[0] == 0) and lse[0] == -np.inf and np.all(p[0] == 0)
    assert np.allclose(out[1], v[0]) and np.allclose(lse[1], q[1] @ k[0] * 0.5 * la.LOG2E)
    assert np.allclose(p[2].sum(), 1.0)
    with pytest.raises(AssertionError):  # a planted mistake: one key fewer
        assert np.allclose(out[2], la.rows_over_keys(q, k, v, [0, 1, 5], 0.5)[0][2])


def test_decode_pages_and_prefix():
    rng = np.random.default_rng(1)
    ckv, kpe = rng.standard_normal((5 * 64, 8)), rng.standard_normal((5 * 64, 3))
    qn, qp = rng.standard_normal((2, 2, 1, 8)), rng.standard_normal((2, 2, 1, 3))
    table = np.array([[3, 1], [0, -1]])
    res = la.decode(qn, qp, ckv, kpe, table, [70, 1], 0.3)
    slot = [3 * 64 + i for i in range(64)] + [64 + i for i in range(6)]
    z = np.array([qn[0, 1, 0] @ ckv[s] + qp[0, 1, 0] @ kpe[s] for s in slot]) * 0.3
    w = np.exp(z) / np.exp(z).sum()
    assert np.allclose(res[0][0][1], w @ ckv[slot]) and np.allclose(res[0][2][0, 69], 0.0)
    assert res[1][1][0] == -np.inf and np.isfinite(res[1][1][1])
    # a prefix and an own part are the same as one sequence of both
    both = la.decode(qn, qp, ckv, kpe, np.array([[2, 3, 1], [2, 0, 0]]), [64 + 70, 64 + 1], 0.3)
    split = la.decode(qn, qp, ckv, kpe, table, [70, 1], 0.3, prefix_table=[2], prefix_len=64)
    assert np.allclose(both[0][0], split[0][0]) and np.allclose(both[0][1], split[0][1])


def test_kept_keys_against_brute_force():
    rng = np.random.default_rng(2)
    for _ in range(200):
        L = int(rng.integers(0, 30))
        budget = int(rng.integers(1, 25))
        recent = int(rng.integers(0, budget + 1))
        w = rng.integers(0, 4, L).astype(np.float32)
        w[rng.random(L) < 0.1] = np.nan
        got = la.kept_keys(w, L, budget, recent).tolist()
        if L <= budget:
            assert got == list(range(L))
            continue
        left = list(range(L - recent))
        best = []
        for _ in range(budget - recent):
            i = max(left, key=lambda i: (np.isnan(w[i]), 0 if np.isnan(w[i]) else w[i], -i))
            best.append(i)
            left.remove(i)
        assert got == sorted(best) + list(range(L - recent, L))
