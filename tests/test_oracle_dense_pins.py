"""The dense-path oracle against hand examples and exact rational arithmetic (CPU)."""
import math
from fractions import Fraction

import numpy as np

from oracle import dense


def rint(fr):
    """Nearest whole number of a Fraction, ties to even."""
    lo = fr.numerator // fr.denominator
    rest = fr - lo
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and lo % 2):
        return lo + 1
    return lo


def test_quantize_by_hand():
    # peak 254: one code is 2, and 1, 3, -5 are ties that go to the even code
    v = np.array([[254.0, 1.0, 3.0, -5.0, 2.0, -254.0, 0.0]])
    q, s = dense.quantize(v)
    assert q.tolist() == [[127, 0, 2, -2, 1, -127, 0]]
    assert s.tolist() == [2.0]
    q, s = dense.quantize(np.array([[0.0, -0.0], [1.0, np.nan], [np.inf, 1.0]]))
    assert q.tolist() == [[0, 0]] * 3 and s[0] == 0 and np.isnan(s[1:]).all()


def test_quantize_codes_are_those_of_the_exact_quotient():
    rng = np.random.default_rng(0)
    s = rng.standard_normal((6, 200)).astype(np.float32)
    w = rng.standard_normal(200).astype(np.float32)
    q, _ = dense.rmsnorm_quantize(s, w)
    for i in range(6):
        v = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(s[i], w)]
        peak = max(abs(f) for f in v)
        assert q[i].tolist() == [rint(127 * f / peak) for f in v]


def test_rmsnorm_by_hand():
    # s = (3, 4): mean square 12.5; eps 12.5 makes the divisor 5
    q, s = dense.rmsnorm_quantize(np.array([[3.0, 4.0]]), np.array([2.0, 1.0]), eps=12.5)
    assert q.tolist() == [[127, 85]]                     # 4 / 6 of 127 = 84.67
    np.testing.assert_allclose(s, [6.0 / 5.0 / 127.0], rtol=1e-15)


def test_linear_by_hand():
    y = dense.linear_int8([[1, -128, 3]], [0.5], [[2, -128, 0], [0, 1, -1]], [2.0, 4.0])
    assert y.tolist() == [[1.0 * (2 + 16384), 2.0 * -131]]


def test_logprobs_by_hand():
    x = np.array([[math.log(1), math.log(2), math.log(5), -np.inf],
                  [-np.inf] * 4, [0.0, np.nan, 1.0, np.nan], [np.inf, 0.0, 0.0, 0.0], [7.0] * 4])
    lp, h, ids, tlp = dense.token_logprobs(x, np.array([1, 0, 0, -1, 4]), top=3)
    np.testing.assert_allclose(lp[0], math.log(0.25), rtol=1e-15)
    np.testing.assert_allclose(
        h[0], -(1 / 8 * math.log(1 / 8) + 1 / 4 * math.log(1 / 4) + 5 / 8 * math.log(5 / 8)), rtol=1e-15)
    assert lp[1] == -np.inf and h[1] == 0 and np.isnan(lp[2]) and np.isnan(h[2])
    assert lp[3] == 0 and np.isnan(h[3]) and np.isnan(lp[4])
    np.testing.assert_allclose(h[4], math.log(4), rtol=1e-15)
    assert ids.tolist() == [[2, 1, 0], [0, 1, 2], [1, 3, 2], [0, 1, 2], [0, 1, 2]]
    np.testing.assert_allclose(tlp[0], np.log([5 / 8, 1 / 4, 1 / 8]), rtol=1e-15)
