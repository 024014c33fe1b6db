"""The numbers with error bounds of bounded.py on the GPU, for sizes that numpy
is too slow for: `v`, `e` and `m` are float64 CUDA tensors.  The kernels add up
a block's rows one after the other, so a sum over rows (axis 0) counts
`row_steps` additions, which the tests derive from the launch; sums within a row
count what they do there."""
import numpy as np
import torch

from bounded import SUM_STEPS, U


class Bounded:
    row_steps = SUM_STEPS

    def __init__(self, v, e=None, m=None):
        self.v = v
        self.e = torch.zeros_like(v) if e is None else e
        self.m = v.abs() + self.e if m is None else m

    @classmethod
    def of(cls, t):
        """Of a tensor, or of numpy numbers with bounds."""
        if isinstance(t, torch.Tensor):
            return cls(t.detach().double())
        return cls(*(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (t.v, t.e, t.m)))

    @property
    def shape(self):
        return tuple(self.v.shape)

    def _other(self, o):
        return o if isinstance(o, Bounded) else Bounded(torch.full((), float(o), dtype=torch.float64, device=self.v.device))

    def __add__(self, o):
        o = self._other(o)
        m = self.m + o.m
        return Bounded(self.v + o.v, self.e + o.e + U * m, m)

    __radd__ = __add__

    def __sub__(self, o):
        o = self._other(o)
        return Bounded(self.v - o.v, self.e + o.e + U * (self.m + o.m))

    def __mul__(self, o):
        o = self._other(o)
        m = self.m * o.m
        return Bounded(self.v * o.v, self.v.abs() * o.e + o.v.abs() * self.e + self.e * o.e + U * m, m)

    __rmul__ = __mul__

    def sum(self, axis, keepdims=False):
        n = int(np.prod([self.shape[a] for a in axis]))
        steps = Bounded.row_steps if 0 in axis else min(n, SUM_STEPS)
        m = self.m.sum(axis, keepdim=keepdims)
        return Bounded(self.v.sum(axis, keepdim=keepdims), self.e.sum(axis, keepdim=keepdims) + steps * U * m, m)

    def mean(self, axis, keepdims=False):
        n = int(np.prod([self.shape[a] for a in axis]))
        s = self.sum(axis, keepdims)
        return Bounded(s.v / n, s.e / n + 4 * U * s.m / n, s.m / n)

    def rsqrt(self):
        low = (self.v - self.e).clamp(min=0.0)
        v = 1.0 / self.v.sqrt()
        e = torch.where(low > 0, 1.0 / low.clamp(min=1e-300).sqrt() - v, float("inf"))
        return Bounded(v, e + 4 * U * (v + e))

    def __getitem__(self, i):
        if isinstance(i, tuple):
            i = tuple(torch.from_numpy(a).to(self.v.device) if isinstance(a, np.ndarray) else a for a in i)
        elif isinstance(i, np.ndarray):
            i = torch.from_numpy(i).to(self.v.device)
        return Bounded(self.v[i], self.e[i], self.m[i])

    def reshape(self, *s):
        return Bounded(self.v.reshape(*s), self.e.reshape(*s), self.m.reshape(*s))

    def joined(self, o):
        return Bounded(*(torch.cat([a, b], -1) for a, b in ((self.v, o.v), (self.e, o.e), (self.m, o.m))))

    def plus(self, o):
        """Two parts of one sum over rows: no rounding of its own."""
        return Bounded(self.v + o.v, self.e + o.e, self.m + o.m)


def check(got, ref, what):
    """|got - ref| within the bound plus one rounding to got's type (and one
    least subnormal, where the value itself underflows)."""
    f = torch.finfo(got.dtype)
    g = got.detach().double()
    assert tuple(g.shape) == ref.shape, (what, g.shape, ref.shape)
    tol = (ref.e + f.eps / 2 * (ref.v.abs() + ref.e)) * (1 + 1e-6) + f.tiny * f.eps
    err = (g - ref.v).abs()
    assert bool(g.isfinite().all()), what
    bad = err > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol).max()), bad.nonzero()[:3].tolist())
