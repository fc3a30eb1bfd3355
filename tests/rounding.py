"""Values with a bound on how far a float32 computation of them may be off.

``Val(v, e)`` holds the float64 value of an expression and a bound on the error
of the same expression in float32: every operation passes its operands' errors
on, with their absolute values, and adds its own rounding, off by at most
f = 2^-24 of the result (half a step) or half the smallest subnormal.  A sum of n
terms in any order is off by at most (n - 1) f times the sum of their
absolute values; sums over a row's columns are trees of a depth that `depth`
bounds.  An expression that fuses a product and a sum rounds once less than
what is counted here.
"""
import numpy as np

F = 2.0 ** -24
TINY = 2.0 ** -150


class Val:
    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def _round(self, v, e):
        return Val(v, e + F * (np.abs(v) + e) + TINY)

    def __add__(self, o):
        o = o if isinstance(o, Val) else Val(o)
        return self._round(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        o = o if isinstance(o, Val) else Val(o)
        return self._round(self.v - o.v, self.e + o.e)

    def __mul__(self, o):
        o = o if isinstance(o, Val) else Val(o)
        return self._round(self.v * o.v,
                           np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    def sum(self, axis, depth, keepdims=False):
        return Val(self.v.sum(axis, keepdims=keepdims),
                   self.e.sum(axis, keepdims=keepdims) * (1 + depth * F) +
                   depth * F * np.abs(self.v).sum(axis, keepdims=keepdims) + TINY)

    def mean(self, depth):
        """Over the columns of a row."""
        n = self.v.shape[-1]
        return self.sum(-1, depth, keepdims=True) * Val(1.0 / n, F / n)

    def rsqrt(self):
        """1 / sqrt of a positive value: a rounded root and a rounded quotient."""
        r = 1.0 / np.sqrt(self.v)
        with np.errstate(divide="ignore", invalid="ignore"):
            lo = np.where(self.e < self.v, 1.0 / np.sqrt(np.maximum(self.v - self.e, 0.0)), np.inf)
        return Val(r, (lo - r) + 3 * F * lo)

    def rounded(self, u, tiny):
        """Stored in a type of half step `u` with half a subnormal `tiny`."""
        return Val(self.v, self.e + u * (np.abs(self.v) + self.e) + tiny)
