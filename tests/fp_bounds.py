"""First-order rounding bounds of fp32 formulas: values in float64 that carry a bound on the error an fp32 evaluation of
the same formula makes, one rounding (u = 2^-24) per operation, sums by their number of additions in a row."""

import numpy as np

U = 2.0 ** -24


class Err:
    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape)

    @staticmethod
    def of(x):
        return x if isinstance(x, Err) else Err(x)

    def __mul__(self, o):
        o = Err.of(o)
        v = self.v * o.v
        return Err(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e + U * np.abs(v))

    __rmul__ = __mul__

    def __add__(self, o):
        o = Err.of(o)
        v = self.v + o.v
        return Err(v, self.e + o.e + U * (np.abs(v) + self.e + o.e))

    __radd__ = __add__

    def __neg__(self):
        return Err(-self.v, self.e)

    def __sub__(self, o):
        return self + (-Err.of(o))

    def sum(self, axis, serial, keepdims=False):
        """A sum in which no term goes through more than `serial` additions."""
        v = self.v.sum(axis, keepdims=keepdims)
        return Err(v, (self.e + serial * U * (np.abs(self.v) + self.e)).sum(axis, keepdims=keepdims))

    def rsqrt(self):
        """v^-1/2 by the hardware instruction (1 ulp = 2 u)."""
        v = self.v ** -0.5
        return Err(v, v * (0.5 * self.e / self.v + 2 * U))

    def sigmoid(self, plain_exp):
        """(s, 1 - s) from e^-|z|: exp2 and reciprocal 1 ulp each, argument, sum and product; with plain_exp the exp2
        argument is the rounded product, wrong by |z| u more."""
        from oracle.sequence import sigmoid
        s, c = sigmoid(self.v), sigmoid(-self.v)
        rel = (7 + (np.abs(self.v) if plain_exp else 0)) * U
        return Err(s, s * rel + s * c * self.e), Err(c, c * rel + s * c * self.e)


def assert_within(name, got, ref, half, tiny=1e-36):
    """got (float64 array) within ref's bound plus the rounding to its type (half steps relative)."""
    err = np.abs(got - ref.v)
    tol = ref.e + half * (np.abs(ref.v) + ref.e) + tiny
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {err.size} outside, worst {np.nanmax(err / tol):.3g} of the bound"
