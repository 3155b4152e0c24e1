"""Pins of the AdamW oracle: torch's own optimizer on the CPU, closed forms of the 8-bit averages, the rounding's mean."""
import numpy as np
import pytest

from oracle import adamw as oa

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_step_matches_torch(wd):
    rng = np.random.default_rng(1)
    w = rng.standard_normal(50)
    p = torch.nn.Parameter(torch.tensor(w, dtype=torch.float64))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.95), eps=1e-8, weight_decay=wd, foreach=False)
    m, v = np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.tensor(g)
        opt.step()
        w, m, v = oa.step(w, g, m, v, 0.01, 0.9, 0.95, 1e-8, t, wd)
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_codes_stand_for_what_the_formula_says():
    m = oa.decode(np.array([-127, -64, 0, 1, 127], dtype=np.int8), [2.0], "m")
    np.testing.assert_allclose(m, 2.0 * np.array([-1.0, -(64 / 127) ** 2, 0.0, 127.0 ** -2, 1.0]), rtol=4 * 2.0 ** -24)
    v = oa.decode(np.array([0, 1, 128, 255], dtype=np.uint8), [3.0], "v")
    np.testing.assert_allclose(v, 3.0 * (np.array([0, 1, 128, 255]) / 255.0) ** 4, rtol=6 * 2.0 ** -24)


@pytest.mark.parametrize("which,n", [("m", 1), ("m", 700), ("v", 513)])
def test_nearest_codes_are_a_fixed_point_and_near(which, n):
    rng = np.random.default_rng(n)
    x = (rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n))).astype(np.float32)
    x = np.abs(x) if which == "v" else x
    c, s = oa.encode(x, which)
    y = oa.decode(c, s, which)
    # once more: the levels are their own codes (their scale: the largest is a level)
    c2, s2 = oa.encode(y, which, np.full(n, 0))
    assert np.max(np.abs(c2.astype(int) - c.astype(int))) <= 1
    lev = oa.levels(which).astype(np.float64)
    gap = np.diff(lev)
    cell = np.clip(np.searchsorted(lev, np.abs(x) / np.repeat(s, 256)[:n], side="right") - 1, 0, len(gap) - 1)
    lim = np.repeat(s, 256)[:n] * gap[cell] * (1.0 if which == "v" else 0.5) * (1 + 1e-3) + 1e-6 * np.abs(x)
    assert np.all(np.abs(x.astype(np.float64) - y) <= lim)


def test_edges_of_a_block():
    assert not np.any(oa.encode(np.zeros(300, dtype=np.float32), "m")[0])
    x = np.full(5, 2.0 ** -121, dtype=np.float32)
    c, s = oa.encode(x, "v")
    assert not c.any() and not s.any()
    v = np.array([1.0, 1e-30, 0.0], dtype=np.float32)
    assert oa.encode(v, "v")[0].tolist() == [255, 1, 0]  # a v above 0 keeps a code above 0
    assert oa.encode(np.array([1.0, 1e-30, -0.9], dtype=np.float32), "m")[0].tolist() == [127, 0, -120]


def test_rounding_by_chance_keeps_the_mean():
    """One value, n different chances: the mean of n numbers with a spread of one gap is off by gap / sqrt(n) at most
    half (standard deviation of one coin throw: gap / 2); six of these are allowed."""
    n = 256 * 400
    bits, more = oa.random_bits(np.arange(n), 7, 3)
    for which, r, val in (("m", bits & np.uint64(0xffff), 0.3337), ("v", bits >> np.uint64(16), 0.2221)):
        x = np.full(n, val, dtype=np.float32)
        x[::256] = 1.0  # the block's scale
        c, s = oa.encode(x, which, r)
        y = oa.decode(c, s, which).reshape(-1, 256)[:, 1:]
        lev = oa.levels(which).astype(np.float64)
        gap = np.diff(lev)[np.searchsorted(lev, val) - 1]
        assert abs(y.mean(dtype=np.float64) - val) <= 6 * 0.5 * gap / np.sqrt(y.size) + 2.0 ** -16 * gap
        assert len(np.unique(y)) == 2
    # uniform in each of 16 parts, for the three numbers and for three keys: 6 deviations of a count
    for seed, step in ((7, 3), (7, 4), (0, 1)):
        bits, more = oa.random_bits(np.arange(n), seed, step)
        for u in (bits & np.uint64(0xffff), bits >> np.uint64(16), more):
            h = np.bincount((u >> np.uint64(12)).astype(int), minlength=16)
            assert np.all(np.abs(h - n / 16) <= 6 * np.sqrt(n / 16))


def test_places_start_at_blocks():
    p = oa.places([1, 256, 257, 0, 3])
    assert [a[0] if len(a) else None for a in p] == [0, 256, 512, None, 1024]
