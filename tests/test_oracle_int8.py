"""Pins of the 8-bit integer oracle (no GPU)."""
import numpy as np

import oracle
from oracle import int8 as oi8


def test_codes_by_hand():
    # amax 127: the multiplier is 1 and the codes are the values, halves to even
    q, s = oi8.quantize_rows(np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, 3.4, 0.0]], dtype=np.float32))
    assert q.tolist() == [[127, -127, 0, 2, 2, 0, 3, 0]] and s.tolist() == [1.0]
    q, s = oi8.quantize_rows(np.array([[0.0, -0.0], [4.0, -2.0], [np.inf, 1.0], [1.0, np.nan], [1e-38, 0.0]], dtype=np.float32))
    assert q.tolist() == [[0, 0], [127, -64], [0, 0], [0, 0], [0, 0]]  # 63.5 goes to the even 64
    assert s[0] == 1 and s[1] == np.float32(4) / np.float32(127) and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 1


def test_quantisation_is_within_half_a_step():
    a = np.random.default_rng(1).standard_normal((50, 300)).astype(np.float32)
    q, s = oi8.quantize_rows(a)
    # half a step, and two FP32 roundings of a value of at most 127 steps
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - a) <= s[:, None] * (0.5 + 127 * 2.0 ** -22))
    assert np.all(np.abs(q).max(axis=1) == 127)


def test_matmul_groups():
    rng = np.random.default_rng(2)
    x, w = rng.integers(-127, 128, (9, 64)).astype(np.int8), rng.integers(-127, 128, (3, 8, 64)).astype(np.int8)
    xs, ws = rng.random(9).astype(np.float32), rng.random((3, 8)).astype(np.float32)
    y = oi8.matmul(x, xs, w, ws, [1, 4, 4, 8])
    assert np.isnan(y[[0, 8]]).all()
    for r, g in ((1, 0), (3, 0), (4, 2), (7, 2)):
        for o in range(8):
            want = int(x[r].astype(int) @ w[g, o].astype(int)) * float(xs[r]) * float(ws[g, o])
            np.testing.assert_allclose(y[r, o], want, rtol=1e-14)


def test_forward_is_near_the_unquantised_layer():
    rng = np.random.default_rng(3)
    T, H, I, E, k = 40, 128, 64, 8, 2
    x, lg = rng.standard_normal((T, H)).astype(np.float32), rng.standard_normal((T, E)).astype(np.float32)
    w1, w2 = (rng.standard_normal(s).astype(np.float32) * 0.1 for s in ((E, 2 * I, H), (E, H, I)))
    P_c, _ = oracle.required_extent(T, k, E, 1)
    kw = dict(k=k, e0=0, E_local=E, n_chunks=1, P_c=P_c)
    got = oi8.forward(x, lg, *oi8.quantize_rows(w1), *oi8.quantize_rows(w2), **kw)
    want = oracle.forward(x, lg, w1, w2, **kw)["out"]
    # each of the four quantisations is off by up to half of amax / 127, about 1% of an element's size
    assert np.linalg.norm(got["out"] - want) <= 0.04 * np.linalg.norm(want)


def test_rows_between_the_experts_and_combine_decode():
    c = np.array([0x0000, 0x8000, 0x0001, 0x00ff, 0x0100, 0x3f00, 0xbf80, 0x4001, 0x7ffe, 0x7fff, 0xffff], np.uint16)
    want = [0.0, 0.0, 2.0 ** -70, 255 * 2.0 ** -70, 2.0 ** -62, 1.0, -1.5, 2.0 + 2.0 ** -7, 2.0 ** 65 - 2.0 ** 57, np.nan, np.nan]
    np.testing.assert_array_equal(oi8.decode_yd(c.view(np.int16)), want)
