"""Pins of the router-loss oracle: brute force, closed forms and finite differences (no GPU)."""
import numpy as np
import pytest

from oracle import router_loss as orl


def _draw(T, E, k, seed):
    rng = np.random.default_rng(seed)
    lg = rng.standard_normal((T, E))
    return lg, np.argsort(-lg, axis=1, kind="stable")[:, :k], rng


def test_loss_matches_a_token_by_token_sum():
    T, E, k = 37, 6, 2
    lg, idx, rng = _draw(T, E, k, 1)
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    off = [3, 10, 10, 30]
    f = orl.router_loss(lg, idx, k, 0.3, 0.7, off, mask)
    bal, z, n, full = 0.0, 0.0, 0, 0
    for s in range(3):
        cnt, pr, ns = [0.0] * E, [0.0] * E, 0
        for t in range(off[s], off[s + 1]):
            if not mask[t]:
                continue
            ns += 1
            den = sum(np.exp(v) for v in lg[t])
            z += np.log(den) ** 2
            for e in range(E):
                pr[e] += np.exp(lg[t, e]) / den
            for e in idx[t]:
                cnt[e] += 1
        assert list(f["seg_counts"][s]) == cnt and f["seg_tokens"][s] == ns
        if ns:
            full, n = full + 1, n + ns
            bal += E * sum(c / (ns * k) * p / ns for c, p in zip(cnt, pr))
    np.testing.assert_allclose(f["loss"], [0.3 * bal / full + 0.7 * z / n, bal / full, z / n], rtol=1e-12)
    assert list(f["seg_tokens"][3:]) == [n, full]


def test_balanced_load_gives_one_and_no_gradient():
    E, k = 8, 2
    idx = np.array([[(t * k + j) % E for j in range(k)] for t in range(E)])
    f = orl.router_loss(np.zeros((E, E)), idx, k, 1.0, 0.0)
    np.testing.assert_allclose(f["loss"][1], 1.0, rtol=1e-14)
    np.testing.assert_allclose(orl.router_loss_bwd(f, k, 1.0, 0.0), 0.0, atol=1e-16)


@pytest.mark.parametrize("off,masked", [(None, False), ([0, 5, 5, 11], True), ([2, 9], False)])
def test_gradient_matches_differences(off, masked):
    T, E, k = 12, 7, 3
    lg, idx, rng = _draw(T, E, k, 2)
    mask = (rng.random(T) < 0.6).astype(np.uint8) if masked else None
    a, b, g = 0.8, 0.05, 1.7
    grad = orl.router_loss_bwd(orl.router_loss(lg, idx, k, a, b, off, mask), k, a, b, g)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = lg.copy(), lg.copy()
            up[t, e] += h
            dn[t, e] -= h
            d = (orl.router_loss(up, idx, k, a, b, off, mask)["loss"][0] -
                 orl.router_loss(dn, idx, k, a, b, off, mask)["loss"][0]) / (2 * h)
            # central difference: h^2 truncation and eps / h rounding, both near 1e-9 here
            assert abs(g * d - grad[t, e]) <= 1e-8


def test_left_out_rows_reach_nothing():
    T, E, k = 9, 4, 2
    lg, idx, _ = _draw(T, E, k, 3)
    mask = np.ones(T, dtype=np.uint8)
    mask[4] = 0
    bad = lg.copy()
    bad[4] = np.nan      # masked
    bad[0] = np.inf      # before the first segment
    bad[6] = -np.inf     # no finite logit
    f = orl.router_loss(bad, idx, k, 1.0, 1.0, [1, T], mask)
    keep = [1, 2, 3, 5, 7, 8]
    ref = orl.router_loss(lg[keep], idx[keep], k, 1.0, 1.0)
    np.testing.assert_allclose(f["loss"], ref["loss"], rtol=1e-13)
    assert not np.any(orl.router_loss_bwd(f, k, 1.0, 1.0)[[0, 4, 6]])
    assert not np.any(f["lse"][[0, 4, 6]])
