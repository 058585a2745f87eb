"""Pins of the fp64 definitions in oracle/lm.py: rows worked out by hand,
finite differences, and mistakes that a wrong definition would make."""
import math

import numpy as np
import pytest

from oracle import lm as L


def test_log_probs_of_rows_by_hand():
    ln2 = math.log(2.0)
    x = np.array([[0.0, ln2, ln2, -np.inf], [5.0, 5.0, 5.0, 5.0], [-np.inf] * 4, [0.0, 0.0, -np.inf, -np.inf]])
    r = L.log_probs(x, np.array([1, 0, 2, -1]), 1.0, 4)
    # row 0: weights 1, 2, 2, 0 of 5
    assert r["logp"][0] == pytest.approx(math.log(0.4)) and r["lse"][0] == pytest.approx(math.log(5.0))
    assert r["entropy"][0] == pytest.approx(-(0.2 * math.log(0.2) + 0.8 * math.log(0.4)))
    assert r["top_ids"][0].tolist() == [1, 2, 0, 3] and r["top_logp"][0][3] == -math.inf
    assert r["logp"][1] == pytest.approx(-math.log(4.0)) and r["entropy"][1] == pytest.approx(math.log(4.0))
    assert r["top_ids"][1].tolist() == [0, 1, 2, 3]
    assert r["lse"][2] == r["logp"][2] == -math.inf and r["entropy"][2] == 0.0
    assert r["logp"][3] == 0.0 and r["entropy"][3] == pytest.approx(ln2)
    # scale 2: weights 1, 4, 4
    r = L.log_probs(x[:1], np.array([0]), 2.0)
    assert r["logp"][0] == pytest.approx(-math.log(9.0)) and r["row_max"][0] == ln2


def test_ordering_of_zeros_and_nan():
    assert L.top_indices(np.array([-0.0, 0.0, np.nan, 1.0, np.nan]), 5).tolist() == [2, 4, 3, 0, 1]
    r = L.log_probs(np.array([[0.0, np.nan], [0.0, np.inf]]), np.array([0, 0]))
    assert np.isnan(r["logp"]).all() and np.isnan(r["entropy"]).all() and r["row_max"][1] == np.inf


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_log_prob_gradient_against_differences(scale):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 9)) * 3
    x[1, [2, 5]] = -np.inf
    t = np.array([3, 0, -1, 8])
    g, h, l = rng.standard_normal((3, 4))

    def loss(y):
        r = L.log_probs(y, t, scale)
        return float((g * r["logp"] + h * r["entropy"] + l * r["lse"]).sum())

    d = L.log_probs_backward(x, t, g, h, l, scale)
    for i in range(4):
        for j in range(9):
            if x[i, j] == -np.inf:
                assert d[i, j] == 0.0
                continue
            a, b = x.copy(), x.copy()
            a[i, j] += 1e-5
            b[i, j] -= 1e-5
            assert d[i, j] == pytest.approx((loss(a) - loss(b)) / 2e-5, abs=2e-9)
    # the entropy's gradient without "+ entropy" (a plausible mistake) would not sum to zero
    assert abs(L.log_probs_backward(x, t, 0 * g, h, None, scale).sum(1)).max() < 1e-12


def test_embedding_and_gradient_are_adjoint():
    rng = np.random.default_rng(6)
    w, g = rng.integers(-8, 9, (5, 3)).astype(float), rng.integers(-8, 9, (7, 3)).astype(float)  # sums are exact
    t = np.array([4, 0, 4, -1, 9, 2, 4])
    out = L.embedding(w, t, 2.0)
    assert np.array_equal(out[0], 2.0 * w[4]) and not out[3].any() and not out[4].any()
    d, a = L.embedding_backward(g, t, 5, 2.0)
    assert float((out * g).sum()) == pytest.approx(float((w * d).sum()))
    assert np.array_equal(d[4], 2 * (g[0] + g[2] + g[6])) and not d[1].any() and not d[3].any()
    assert np.array_equal(L.embedding_backward(g, t, 5, 2.0, w)[0], w + d) and (a >= np.abs(d)).all()


def test_clip_by_hand():
    norm, c, norms, out = L.clip_grads([np.array([3.0, 0.0]), np.array([[4.0]])], 1.0)
    assert norm == 5.0 and c == 0.2 and norms.tolist() == [3.0, 4.0]
    assert out[1][0, 0] == pytest.approx(0.8)
    assert L.clip_grads([np.array([3.0, 4.0])], 5.0)[1] == 1.0
    assert L.clip_grads([np.array([3.0, np.inf])], 1.0)[1] == 1.0
    assert L.clip_grads([np.zeros(3)], 0.0)[1] == 1.0
