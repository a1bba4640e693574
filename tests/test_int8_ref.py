"""The INT8 and balance references against definitions written another way:
rationals for the rows, a loop for the product, differences for the gradient."""
from fractions import Fraction as Fr

import numpy as np

import balance_ref as B
import int8_ref as R
from oracle import brute


def _rn_int(v):
    f = v.numerator // v.denominator
    r = v - f
    return f + (r > Fr(1, 2) or (r == Fr(1, 2) and f % 2 == 1))


def test_rows_against_rationals():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((7, 48)) * np.exp(rng.uniform(-30, 30, (7, 1)))).astype(np.float32)
    x[1] = 0
    x[2] = np.linspace(-127, 127, 48).astype(np.float32)
    x[3] = np.arange(48) - 0.5
    x[3, 0] = 127                                       # scale 1: halves go to the even code
    x[4, 5] = 1e30
    codes, s = R.quantize(x)
    for i in range(7):
        amax = max(abs(Fr(float(v))) for v in x[i])
        sc = brute.rn32(brute.rn64(amax / 127))
        assert Fr(float(s[i])) == sc
        r = brute.rn32(brute.rn64(1 / sc)) if sc else Fr(0)
        assert codes[i].tolist() == [_rn_int(brute.rn32(Fr(float(v)) * r)) for v in x[i]]
    assert codes[3, :6].tolist() == [127, 0, 2, 2, 4, 4]


def test_rows_out_of_range():
    x = np.ones((4, 16), np.float32)
    x[0, 3], x[1, 4] = np.nan, -np.inf
    x[2] = 1e-45
    x[3] = 3.4e38
    codes, s = R.quantize(x)
    assert np.isnan(s[:2]).all() and not codes[:2].any()
    assert s[2] == np.float32(2.0 ** -126) and not codes[2].any()
    assert (codes[3] == 127).all() and np.isfinite(s[3])


def test_product_against_a_loop():
    rng = np.random.default_rng(4)
    a = rng.integers(-127, 128, (5, 16)).astype(np.int8)
    w = rng.integers(-127, 128, (3, 4, 16)).astype(np.int8)
    sa, sw = rng.random(5).astype(np.float32), rng.random((3, 4)).astype(np.float32)
    off, gat = np.array([0, 2, 2, 6]), np.array([4, 0, 1, 1, 2, 3])
    y = R.product(a, sa, w, sw, off, gat)
    for j in range(6):
        g = 0 if j < 2 else 2
        for n in range(4):
            acc = sum(int(a[gat[j], k]) * int(w[g, n, k]) for k in range(16))
            assert y[j, n] == np.float32(np.float32(sa[gat[j]] * sw[g, n]) * np.float32(acc))


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((9, 6))
    z[2, 3] = -np.inf
    z[4] = -np.inf
    ids = np.argsort(-z, 1)[:, :2].astype(np.int32)
    ids[7, 1] = -1
    mask = np.ones(9, np.uint8)
    mask[6] = 0
    g = np.array([0.7, -0.3])
    r = B.balance(z, ids, mask, g)
    assert r["tokens"] == 7 and r["counts"].sum() == 13
    h = 1e-6
    for t in range(9):
        for e in range(6):
            if z[t, e] == -np.inf:
                assert r["grad"][t, e] == 0
                continue
            v = []
            for sgn in (1, -1):
                q = z.copy()
                q[t, e] += sgn * h
                v.append((B.balance(q, ids, mask)["losses"] * g).sum())
            assert abs((v[0] - v[1]) / (2 * h) - r["grad"][t, e]) < 1e-8


def test_balance_closed_forms():
    z = np.zeros((8, 4))
    ids = np.array([[0, 1], [2, 3]] * 4, np.int32)
    r = B.balance(z, ids)
    assert abs(r["losses"][0] - 1) < 1e-15 and abs(r["losses"][1] - np.log(4) ** 2) < 1e-15
    z[:, 0] = 100.0
    r = B.balance(z, np.zeros((8, 1), np.int32))        # everything on one expert
    assert abs(r["losses"][0] - 4) < 1e-12
    r = B.balance(np.full((3, 4), -np.inf), np.zeros((3, 2), np.int32), None, [1, 1])
    assert r["tokens"] == 0 and not r["losses"].any() and not r["grad"].any()
