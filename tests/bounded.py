"""Numbers with a bound on the error that float32 arithmetic may have made of
them (running error analysis): `v` the float64 value, `e` the bound, `m` the
sum of the magnitudes of the terms that the value is made of.  An operation
adds half a step (2^-24) of its magnitude and what its operands' bounds grow
to.  Taking the magnitude of the terms and not of the result lets the kernels
multiply out what the definition has in brackets; a difference is formed by
both, so its terms end there.  A sum of n values in any order adds at most
min(n, SUM_STEPS) half steps of the sum of magnitudes, SUM_STEPS being the
longest chain of additions in the kernels on the tests' sizes: up to 32 values
of a thread (or rows of a block), 5 shuffles, 32 warps.  Divisions, reciprocal
roots, sines and cosines count 4 half steps (CUDA's documented errors of at
most 2 units in the last place)."""
import numpy as np

U = 2.0 ** -24
SUM_STEPS = 32 + 5 + 32


class Bounded:
    __array_ufunc__ = None

    def __init__(self, v, e=None, m=None):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.zeros_like(self.v) if e is None else e
        self.m = np.abs(self.v) + self.e if m is None else m

    @property
    def shape(self):
        return self.v.shape

    @staticmethod
    def of(o):
        return o if isinstance(o, Bounded) else Bounded(o)

    def __add__(self, o):
        o = Bounded.of(o)
        m = self.m + o.m
        return Bounded(self.v + o.v, self.e + o.e + U * m, m)

    __radd__ = __add__

    def __sub__(self, o):
        o = Bounded.of(o)
        return Bounded(self.v - o.v, self.e + o.e + U * (self.m + o.m))

    def __rsub__(self, o):
        return Bounded.of(o) - self

    def __mul__(self, o):
        o = Bounded.of(o)
        m = self.m * o.m
        return Bounded(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e + U * m, m)

    __rmul__ = __mul__

    def sum(self, axis, keepdims=False):
        n = int(np.prod([self.shape[a] for a in axis]))
        m = self.m.sum(axis=axis, keepdims=keepdims)
        return Bounded(self.v.sum(axis=axis, keepdims=keepdims),
                       self.e.sum(axis=axis, keepdims=keepdims) + min(n, SUM_STEPS) * U * m, m)

    def mean(self, axis, keepdims=False):
        n = int(np.prod([self.shape[a] for a in axis]))
        s = self.sum(axis, keepdims)
        return Bounded(s.v / n, s.e / n + 4 * U * s.m / n, s.m / n)

    def rsqrt(self):
        low = np.maximum(self.v - self.e, 0.0)
        with np.errstate(divide="ignore", invalid="ignore"):
            v = 1.0 / np.sqrt(self.v)
            e = np.where(low > 0, 1.0 / np.sqrt(np.maximum(low, 1e-300)) - v, np.inf)
        return Bounded(v, e + 4 * U * (v + e))

    def __getitem__(self, i):
        return Bounded(self.v[i], self.e[i], self.m[i])

    def reshape(self, *s):
        return Bounded(self.v.reshape(*s), self.e.reshape(*s), self.m.reshape(*s))

    def joined(self, o):
        return Bounded(*(np.concatenate([a, b], -1) for a, b in ((self.v, o.v), (self.e, o.e), (self.m, o.m))))


def turned(cos, sin, positions, freq):
    """Cosines and sines as the kernels form them: the turns of a position in
    float64 (three roundings), the rest below half a turn rounded to float32
    (2^-26 of a turn), the functions within 4 half steps."""
    turns = np.abs(positions).max(initial=0) * np.abs(freq).max(initial=0) / (2 * np.pi)
    off = 2 * np.pi * (2.0 ** -26 + 3 * 2.0 ** -53 * turns) + 2.0 ** -52 * 2 * np.pi * turns
    return tuple(Bounded(t, off + 4 * U * (np.abs(t) + off)) for t in (cos, sin))


def check(got, ref, what):
    """|got - ref| within the bound plus one rounding to got's type (and one
    least subnormal, where the value itself underflows)."""
    import torch
    h = torch.finfo(got.dtype).eps / 2
    g = got.detach().double().cpu().numpy()
    ref = Bounded.of(ref)
    assert g.shape == ref.v.shape, (what, g.shape, ref.v.shape)
    tiny = torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps
    tol = (ref.e + h * (np.abs(ref.v) + ref.e)) * (1 + 1e-6) + tiny
    err = np.abs(g - ref.v)
    assert np.isfinite(g).all(), what
    bad = err > tol
    assert not bad.any(), (what, int(bad.sum()), float((err / tol).max()), np.argwhere(bad)[:3].tolist())
