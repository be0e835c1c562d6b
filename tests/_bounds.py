"""Running error analysis for the GPU tests: a value in float64 beside a bound
on how far a float32 computation of it may be off.

Every operation adds one rounding of at most ROUND = 2^-24 of its result to
what its operands bring (products: |a| e_b + |b| e_a + e_a e_b).  A sum of n
terms in an order that is not known has n - 1 roundings at most, each of a
partial sum of at most the sum of the terms' magnitudes.  Functions bring their
own relative error and their slope times the argument's.
"""
import numpy as np

ROUND = 2.0 ** -24
EX2 = 2.0 ** -21   # an exponential: 2^-22.7 measured for its base-2 form over [-8, 0], 2^-22 and a rounding beyond
LEAST = 2.0 ** -110  # what float32 may lose to underflow of a factor, with the others below 2^16


class R:
    """A real number (array) and its bound."""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def __getitem__(self, i):
        return R(self.v[i], self.e[i])

    def _rounded(self, v, e):
        return R(v, e * (1 + ROUND) + ROUND * np.abs(v))

    def __mul__(self, o):
        o = o if isinstance(o, R) else R(o)
        return self._rounded(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    def __add__(self, o):
        o = o if isinstance(o, R) else R(o)
        return self._rounded(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        o = o if isinstance(o, R) else R(o)
        return self._rounded(self.v - o.v, self.e + o.e)

    def sum(self, axis, terms=None):
        n = self.v.shape[axis] if terms is None else terms
        return R(self.v.sum(axis), (self.e + n * ROUND * (np.abs(self.v) + self.e)).sum(axis))

    def exp(self):
        # base 2: the product with log2 e rounds the argument by |x| 2^-24, its constant by as much
        v = np.exp(self.v)
        return R(v, v * (np.expm1(self.e + 2 * ROUND * np.abs(self.v)) + EX2))

    def sigmoid(self):
        s = 1 / (1 + np.exp(-self.v))
        # exp(-x) is off by e + 2 |x| 2^-24 + EX2 of itself, the quotient by 1 - s of that and two roundings
        return R(s, s * ((1 - s) * (np.expm1(self.e + 2 * ROUND * np.abs(self.v)) + EX2) + 4 * ROUND))

    def softplus(self):
        v = np.logaddexp(self.v, 0)
        return R(v, 1.01 * self.e * np.minimum(1.0, v) + v * 2.0 ** -20)  # its slope, a sigmoid, is below 1 and below v


def silu(u):
    return u * u.sigmoid()


def silu_slope(u):
    s = u.sigmoid()
    return s * (u * (R(np.ones_like(s.v)) - s) + 1.0)


def close(got, want, half, name):
    """Each element within its bound and one rounding of `half` of the value to the output's type."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.v.shape, (name, got.shape, want.v.shape)
    tol = half * (np.abs(want.v) + want.e) + want.e + LEAST
    bad = ~(np.abs(got - want.v) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} for "
                           f"{want.v[bad][0]}, tolerance {tol[bad][0]}")
