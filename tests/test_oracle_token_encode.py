"""The float64 oracle of the encoding and tree operators against hand-computed numbers, closed forms and brute force."""
import math

import numpy as np
import pytest
import torch

from oracle import latent_attention as la
from oracle import token_encode as te


def test_norms_by_hand():
    x = np.array([1.0, 3.0])
    y, reach = te.layer_norm(x, np.array([2.0, 1.0]), np.array([0.5, 0.0]), 3.0)
    assert np.allclose(y, [-2.0 / 2.0 + 0.5, 1.0 / 2.0])  # mean 2, variance 1, sqrt(1 + 3) = 2
    assert np.allclose(reach, [3.0 / 2.0 * 2.0 + 0.5, 5.0 / 2.0])
    assert np.allclose(te.rms_norm(x, np.array([1.0, 2.0]), 4.0), [1.0 / 3.0, 2.0])  # mean square 5


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_one_of_complex_numbers(interleaved):
    rng = np.random.default_rng(0)
    x, angle = rng.standard_normal((5, 64)), rng.standard_normal((5, 32))
    y = te.rotate(x, np.concatenate([np.cos(angle), np.sin(angle)], -1), interleaved)
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * angle[:, i])
        assert np.allclose(y[:, a], z.real) and np.allclose(y[:, b], z.imag)


def test_hadamard_by_hand_and_its_inverse():
    assert np.allclose(te.hadamard(4) * 2, [[1, 1, 1, 1], [1, -1, 1, -1], [1, 1, -1, -1], [1, -1, -1, 1]])
    h = te.hadamard(128)
    assert np.allclose(h @ h, np.eye(128)) and np.allclose(h, h.T)


def test_nearest_codes_against_torch():
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.standard_normal(20000) * s for s in (0.001, 0.02, 1, 30, 100)])
    v = np.clip(np.concatenate([v, te.values(np.arange(127)), -te.values(np.arange(127)), [0.0, 448.0]]), -448, 448)
    ties = (te.values(np.arange(126)) + te.values(np.arange(1, 127))) / 2  # exact in fp32
    v = np.concatenate([v, ties, -ties]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(te.nearest_codes(v.astype(np.float64)), want)


def test_rows_scales_and_reach():
    rng = np.random.default_rng(2)
    x, angle = rng.standard_normal((3, 2, 128)), rng.standard_normal((3, 32))
    cs = np.concatenate([np.cos(angle), np.sin(angle)], -1)
    norm = (rng.standard_normal(128), rng.standard_normal(128), 1e-6)
    for n in (None, norm):
        for had in (False, True):
            for inter in (False, True):
                y, reach = te.index_rows(x, cs, n, inter, had)
                assert np.all(np.abs(y) <= reach * (1 + 1e-12))
                base = te.layer_norm(x, *n)[0] if n else x
                # every step but the norm keeps a row's length
                assert np.allclose((y ** 2).sum(-1), (base ** 2).sum(-1))
                assert np.allclose(te.scales(y), np.abs(y).max((1, 2)) / 448)
    assert np.array_equal(te.scales(np.zeros((2, 1, 128))), [1.0, 1.0])
    with pytest.raises(AssertionError):  # a planted mistake: the other order of pairs
        assert np.allclose(te.index_rows(x, cs, None, True, False)[0], te.index_rows(x, cs, None, False, False)[0])


def test_a_chain_is_a_tree():
    """Nodes that see all nodes up to themselves are the tokens of a decode step."""
    rng = np.random.default_rng(3)
    ckv, kpe = rng.standard_normal((4 * 64, 8)), rng.standard_normal((4 * 64, 3))
    qn, qp = rng.standard_normal((2, 3, 2, 8)), rng.standard_normal((2, 3, 2, 3))
    table = np.array([[3, 1], [0, -1]])
    chain = la.decode(qn, qp, ckv, kpe, table, [70, 3], 0.3)
    tree = la.tree(qn, qp, ckv, kpe, table, [70, 3], [[set(range(i + 1)) for i in range(3)]] * 2, 0.3)
    for a, b in zip(chain, tree):
        assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_a_tree_by_hand():
    """Two nodes behind one key; the second does not see the first, the third query is padding."""
    ckv = np.array([[1.0], [2.0], [4.0]] + [[np.nan]] * 61)
    kpe, qp = np.zeros((64, 1)), np.zeros((1, 3, 1, 1))
    qn = np.ones((1, 3, 1, 1))
    (out, lse, p, _, _), = la.tree(qn, qp, ckv, kpe, np.array([[0]]), [3], [[{0}, {1}]], 1.0)
    e = math.e
    assert np.allclose(p, [[1 / (1 + e), e / (1 + e), 0], [1 / (1 + e ** 3), 0, e ** 3 / (1 + e ** 3)], [0, 0, 0]])
    assert np.allclose(out[:, 0], [(1 + 2 * e) / (1 + e), (1 + 4 * e ** 3) / (1 + e ** 3), 0])
    assert lse[2] == -np.inf
