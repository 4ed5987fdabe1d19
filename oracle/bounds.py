"""Running error bounds: a value's magnitude and how far an fp32 evaluation of it may be off, carried through products and
sums.  ``Bound(m, e)`` stands for a number of absolute value at most m, off by at most e.  A product and a sum add one
rounding each of half a step, 2^-24 of the magnitude; a sum of n terms adds n of them, whatever its order.  First order:
products of two errors are left out."""
import numpy as np

U = 2.0 ** -24


class Bound:
    __array_priority__ = 100.0

    def __init__(self, m, e=0.0):
        self.m = np.abs(np.asarray(m, dtype=np.float64))
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.m.shape)

    def __add__(self, o):
        o = _of(o)
        m = self.m + o.m
        return Bound(m, self.e + o.e + U * m)

    __radd__ = __add__
    __sub__ = __add__
    __rsub__ = __add__

    def __mul__(self, o):
        o = _of(o)
        m = self.m * o.m
        return Bound(m, self.m * o.e + o.m * self.e + U * m)

    __rmul__ = __mul__

    def __neg__(self):
        return self

    def __getitem__(self, k):
        return Bound(self.m[k], self.e[k])

    def sum(self, axis):
        m = self.m.sum(axis)
        return Bound(m, self.e.sum(axis) + self.m.size // max(m.size, 1) * U * m)

    def reshape(self, *s):
        return Bound(self.m.reshape(*s), self.e.reshape(*s))

    def repeat(self, n, axis):
        return Bound(self.m.repeat(n, axis), self.e.repeat(n, axis))


def _of(x):
    return x if isinstance(x, Bound) else Bound(x)


def stack(xs, axis):
    if isinstance(xs[0], Bound):
        return Bound(np.stack([x.m for x in xs], axis), np.stack([x.e for x in xs], axis))
    return np.stack(xs, axis)


def zeros_like(x):
    return Bound(np.zeros_like(x.m)) if isinstance(x, Bound) else np.zeros_like(x)


def sigmoid(z):
    return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def sigmoid_bound(z, ez=0.0):
    """1 / (1 + exp(-z)): the exponential is within two steps (4 U), the sum rounds once, the quotient is within two steps;
    the slope of the sigmoid times z's own error."""
    s = sigmoid(z)
    return Bound(s, 10 * U * s + s * (1 - s) * ez)


def silu_slope(z):
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def silu_slope_bound(z, ez=0.0):
    s = sigmoid_bound(z, ez)
    return s * (Bound(1.0) + Bound(z, ez) * Bound(1 - s.m, s.e + U))
