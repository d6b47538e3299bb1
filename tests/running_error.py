"""Values in 64 bits that carry a bound on the error of the same computation in
fp32, to first order: every operation passes on the errors of its operands and
adds its own rounding, u = 2^-24 of its result.

A sum over n terms adds (n - 1) u of the sum of their sizes, the bound of any
order of the additions.  exp and the reciprocal root of the hardware are good to
2^-22 of their results; exp's argument is scaled by log2(e) first, whose rounding
counts as the argument's size times 2^-23.  What an operation adds is taken
twice over, which covers the second-order terms that the rules leave out (an
error of an operand times another's, below 2^-10 of the first-order ones here)
and fused operations, whose single rounding is smaller.
"""

import numpy as np

U = 2.0 ** -24


class E:
    """value and error bound, arrays of one shape"""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def __add__(self, o):
        o = wrap(o)
        v = self.v + o.v
        return E(v, self.e + o.e + 2 * U * np.abs(v))

    __radd__ = __add__

    def __neg__(self):
        return E(-self.v, self.e)

    def __sub__(self, o):
        return self + (-wrap(o))

    def __rsub__(self, o):
        return wrap(o) + (-self)

    def __mul__(self, o):
        o = wrap(o)
        v = self.v * o.v
        return E(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e + 2 * U * np.abs(v))

    __rmul__ = __mul__

    def __getitem__(self, i):
        return E(self.v[i], self.e[i])

    def reshape(self, *s):
        return E(self.v.reshape(*s), self.e.reshape(*s))

    def sum(self, axis, keepdims=False):
        axes = (axis,) if isinstance(axis, int) else axis
        n = int(np.prod([self.v.shape[a] for a in axes]))
        size = np.abs(self.v).sum(axis, keepdims=keepdims)
        return E(self.v.sum(axis, keepdims=keepdims), self.e.sum(axis, keepdims=keepdims) + 2 * max(n - 1, 0) * U * size)

    def rsqrt(self):
        v = 1.0 / np.sqrt(self.v)
        return E(v, 0.5 * v / self.v * self.e * 1.01 + 2.0 ** -21 * v)

    def exp(self):
        v = np.exp(self.v)
        return E(v, v * np.expm1(np.minimum(self.e + np.abs(self.v) * 2.0 ** -22, 1.0)) + 2.0 ** -21 * v)

    def sigmoid(self):
        p = 1.0 / (1.0 + np.exp(-self.v))
        # slope p (1 - p); exp's own error enters through 1 - p, the sum's and the reciprocal's are relative to p
        e = p * (1 - p) * (self.e * 1.01 + np.abs(self.v) * 2.0 ** -22 + 2.0 ** -21) + 2.0 ** -21 * p
        return E(p, e)

    def round_to(self, step):
        """Stored with half a step of relative rounding (a bf16: 2^-8); bf16 keeps fp32's exponents, so below their
        normal numbers 2^-133 is left"""
        return E(self.v, self.e + step * (np.abs(self.v) + self.e) + 2.0 ** -133)


def wrap(x):
    return x if isinstance(x, E) else E(x)


def act(a, kind):
    """(act(a), its slope) as E"""
    if kind is None:
        return a, E(np.ones_like(a.v))
    p = a.sigmoid()
    q = p * (1.0 - p)
    if kind == "sigmoid":
        return p, q
    return a * p, a * q + p


def group_norm(x, groups, weight, bias, z, activation, rms, eps, dout=None):
    """The norm (or, with dout, its gradients dx, dz, dweight, dbias) with bounds; float64 arrays [rows, C]."""
    rows, C = x.shape
    d = C // groups
    cut = lambda a: E(a.reshape(rows, groups, d))  # noqa: E731
    shared = next((a.shape[0] == d for a in (weight, bias) if a is not None), True)
    each = lambda a, none: E(np.full((1, 1, d), none) if a is None  # noqa: E731
                             else a.reshape(1, 1 if shared else groups, d))
    w, b, c = each(weight, 1.0), each(bias, 0.0), cut(x)
    if not rms:
        c = c - c.sum(-1, True) * E(1.0 / d, U / d)
    r = ((c * c).sum(-1, True) * E(1.0 / d, U / d) + eps).rsqrt()
    n = c * r
    a = n * w + b
    f, df = act(a if z is None else cut(z), activation)
    if dout is None:
        return (f if z is None else a * f).reshape(rows, C)
    dy = cut(dout)
    da = dy * (df if z is None else f)
    dn = da * w
    dx = dn - n * ((dn * n).sum(-1, True) * E(1.0 / d, U / d))
    if not rms:
        dx = dx - dn.sum(-1, True) * E(1.0 / d, U / d)
    over = (0, 1) if shared else (0,)
    dz = None if z is None else (dy * a * df).reshape(rows, C)
    return (dx * r).reshape(rows, C), dz, (da * n).sum(over).reshape(-1), da.sum(over).reshape(-1)


def causal_conv_bwd(dout, x, weight, bias, activation, norm_dim, norm_channels, eps):
    """One sequence; float64 arrays.  (dx, dweight, dbias) with bounds."""
    L, D = x.shape
    W = weight.shape[1]
    u = np.concatenate([np.zeros((W - 1, D)), x])
    c = E(np.zeros((L, D)) if bias is None else np.tile(bias, (L, 1)))
    for j in range(W):
        c = c + E(weight[:, j] * np.ones((L, 1))) * E(u[j: j + L])
    y, slope = act(c, "silu" if activation else None)
    dy = E(dout)
    if norm_channels:
        h = y[:, :norm_channels].reshape(L, norm_channels // norm_dim, norm_dim)
        g = dy[:, :norm_channels].reshape(L, norm_channels // norm_dim, norm_dim)
        r = ((h * h).sum(-1, True) + eps).rsqrt()
        n = h * r
        g = ((g - n * (n * g).sum(-1, True)) * r).reshape(L, norm_channels)
        dy = E(np.concatenate([g.v, dy.v[:, norm_channels:]], 1), np.concatenate([g.e, dy.e[:, norm_channels:]], 1))
    dc = dy * slope
    dx, dw = E(np.zeros((L, D))), []
    for j in range(W):
        dw.append((dc * E(u[j: j + L])).sum(0))
        back = W - 1 - j
        if back < L:
            pad = lambda a: np.concatenate([a[back:], np.zeros((back, D))])  # noqa: E731
            dx = dx + E(pad(dc.v), pad(dc.e)) * E(weight[:, j] * np.ones((L, 1)))
    return dx, E(np.stack([a.v for a in dw], 1), np.stack([a.e for a in dw], 1)), dc.sum(0)
