"""Pins of the score-routing oracle: token-by-token choice, closed forms, finite differences (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import router_scores as ors


def _brute(logits, bias, k, score, G, tg, top):
    """The choice, one token at a time, by repeated search for the largest."""
    s = ors.scores(logits, score)
    T, E = s.shape
    size, out = E // G, []
    for t in range(T):
        c = [float(np.float32(s[t, e] + (0.0 if bias is None else float(bias[e])))) for e in range(E)]
        rank = []
        for g in range(G):
            best = sorted(c[g * size:(g + 1) * size], reverse=True)[:top]
            rank.append(float(np.float32(sum(best))))
        open_, left = set(), dict(enumerate(rank))
        for _ in range(tg):
            g = max(left, key=lambda i: (left[i], -i))
            open_.add(g)
            del left[g]
        cand = {e: c[e] for e in range(E) if e // size in open_}
        row = []
        for _ in range(k):
            e = max(cand, key=lambda i: (cand[i], -i))
            row.append(e)
            del cand[e]
        out.append(row)
    return np.array(out)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,tg,top,bias", [(8, 2, 1, 1, 1, False), (16, 4, 4, 2, 2, True), (12, 3, 6, 3, 1, True),
                                               (6, 6, 6, 6, 2, True)])
def test_choice_matches_a_search(score, E, k, G, tg, top, bias):
    rng = np.random.default_rng(E + G)
    lg = np.round(rng.standard_normal((60, E)) * 2) / 2  # ties
    b = np.round(rng.standard_normal(E), 1).astype(np.float32) if bias else None
    idx, _ = ors.route(lg, b, k, score, G, tg, top)
    np.testing.assert_array_equal(idx, _brute(lg, b, k, score, G, tg, top))


def test_renormalised_softmax_without_extras_is_plain_routing():
    lg = np.random.default_rng(1).standard_normal((50, 16))
    idx, g = ors.route(lg, None, 3, "softmax")
    want = oracle.route(lg, 3)
    np.testing.assert_array_equal(idx, want[0])
    np.testing.assert_allclose(g, want[1], rtol=1e-13)


def test_bias_moves_the_choice_and_not_the_gates():
    lg = np.array([[2.0, 1.0, 0.0, -1.0]])
    b = np.array([-9.0, 0.0, 0.0, 5.0], dtype=np.float32)
    idx, g = ors.route(lg, b, 2, "sigmoid", renormalize=False, scale=2.0)
    assert idx.tolist() == [[3, 1]]
    np.testing.assert_allclose(g[0], [2 / (1 + np.e), 2 / (1 + np.exp(-1.0))], rtol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_without_values(score):
    inf = np.inf
    lg = np.array([[-inf, -inf, -inf, -inf], [np.nan, 1.0, -inf, 0.0], [inf, 0.0, inf, -5.0]])
    idx, g = ors.route(lg, None, 2, score)
    assert idx[0].tolist() == [0, 1] and g[0].tolist() == [0.0, 0.0]
    assert idx[1].tolist() == [1, 3]
    assert idx[2].tolist() == [0, 2] and g[2].tolist() == [0.5, 0.5]
    _, g = ors.route(lg, None, 2, score, renormalize=False)
    assert g[0].tolist() == [0.0, 0.0] and np.all(np.isfinite(g))
    # a bias that shuts every expert out, or is no number, still leaves a choice
    assert ors.route(lg, np.full(4, -inf), 2, score)[0][1].tolist() == [0, 1]
    assert ors.route(lg, np.array([np.nan, -inf, np.nan, 0.0]), 2, score)[0][1].tolist() == [3, 0]


def test_very_small_sigmoid_scores_keep_their_ratio():
    _, g = ors.route(np.array([[-900.0, -901.0, -1000.0]]), None, 2, "sigmoid")
    np.testing.assert_allclose(g[0], np.array([1.0, np.exp(-1.0)]) / (1 + np.exp(-1.0)), rtol=1e-13)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_matches_differences(score, renorm):
    rng = np.random.default_rng(4)
    T, E, k = 5, 9, 3
    lg, dg = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    idx, _ = ors.route(lg, rng.standard_normal(E), k, score, renormalize=renorm, scale=1.7)
    got = ors.backward(lg, idx, dg, score, renorm, 1.7)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = ((ors.gates(up, idx, score, renorm, 1.7) - ors.gates(dn, idx, score, renorm, 1.7)) * dg).sum() / (2 * h)
            assert abs(d - got[t, e]) <= 1e-8  # h^2 truncation and eps / h rounding
    assert np.all(np.abs(got) <= ors.backward_bound(lg, idx, dg, score, renorm, 1.7) * (1 + 1e-12))


def test_bias_update_by_hand():
    counts = np.array([[5, 1, 2, 0], [1, 1, 2, 0]])  # loads 6 2 4 0, mean 3
    b = np.array([0.5, 0.0, 1.0, -1.0], dtype=np.float32)
    np.testing.assert_array_equal(ors.bias_update(b, counts, 0.25), np.array([0.25, 0.25, 0.75, -0.75], dtype=np.float32))
    np.testing.assert_array_equal(ors.bias_update(b, np.full((1, 4), 7), 0.25), b)
