"""Layer norm and the gated linear recurrence in 64 bits (numpy), with the magnitudes that the
tolerances of layer_ops_ref.tol multiply.

Layer norm.  The deviations h - mu carry the rounding of h = x + r (2^-24 |h|, none without a residual),
the error of the mean (roundings of its sum, made up for by the sum of the deviations, so a few 2^-24
of their mean magnitude) and their own rounding; 1 / sqrt(v + eps) has half the relative error of v, a
sum of squares of them.  So hat is off by a few 2^-24 times (|hat| + 1) plus, with a residual, 2^-24
(|h| + mean |h|) / std: `hat_mag`.  Everything else is products and sums of it."""
import numpy as np


def layernorm(x, r, w, b, eps):
    """-> h, y, magnitude of y"""
    h = x if r is None else x + r
    mid = h - h.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((mid * mid).mean(-1, keepdims=True) + eps)
    hat = mid * rstd
    mag = hat_mag(hat, rstd, None if r is None else np.abs(x) + np.abs(r))
    w, b = (1.0 if w is None else w), (0.0 if b is None else b)
    return h, hat * w + b, mag * np.abs(w) + np.abs(b)


def hat_mag(hat, rstd, h=None):
    m = np.abs(hat) + 1
    return m if h is None else m + (h + h.mean(-1, keepdims=True)) * rstd


def layernorm_back(h, w, dy, dh, eps):
    """-> dict of (value, magnitude)"""
    mid = h - h.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((mid * mid).mean(-1, keepdims=True) + eps)
    hat = mid * rstd
    m = hat_mag(hat, rstd)
    wdy = dy if w is None else dy * w
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    dx = rstd * (wdy - mean(wdy) - hat * mean(wdy * hat))
    dxm = rstd * (np.abs(wdy) + mean(np.abs(wdy)) + m * mean(np.abs(wdy) * m))
    if dh is not None:
        dx, dxm = dx + dh, dxm + np.abs(dh)
    return dict(dx=(dx, dxm), dw=((dy * hat).sum(0), (np.abs(dy) * m).sum(0)), db=(dy.sum(0), np.abs(dy).sum(0)))


def glr(x, r, i, z, lam, rb, ib, c, h0, dy=None, dh=None, mag=False):
    """Gated linear recurrence of one sequence, x, r, i, z [L, D], h0 [D]; with dy the gradients too.  mag: the same on
    absolute values, what a tolerance multiplies: a step adds the rounding of a (2^-24, 2^-22 of 1 - a) times h to
    those of the steps before, gates and u are a few 2^-22 off, so (L + 64) 2^-22 of it covers L steps."""
    a_ = np.abs if mag else (lambda v: v)
    sig = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
    L, D = x.shape
    rate = c * np.logaddexp(lam, 0)
    sr = sig(r + (0 if rb is None else rb))
    si = np.ones_like(x) if i is None else sig(i + (0 if ib is None else ib))
    s = rate * sr
    a, b2 = np.exp(-s), -np.expm1(-2 * s)
    u = np.sqrt(b2) * si * a_(x)
    gate = np.ones_like(x) if z is None else a_(z * sig(z))
    hs = [a_(h0)]
    for t in range(L):
        hs.append(a[t] * hs[-1] + u[t])
    path = np.array(hs)
    out = dict(y=path[1:] * gate, h=path[-1])
    if dy is None:
        return out
    v, before = a_(dy) * gate, path[:-1]
    g, carry = np.zeros_like(x), np.zeros(D) if dh is None else a_(dh)
    for t in reversed(range(L)):
        g[t] = v[t] + carry
        carry = a[t] * g[t]
    q = np.where(s > 0, s / np.where(b2 > 0, b2, 1), 0.5)
    Q = g * (u * a * a * q + (1 if mag else -1) * s * a * before)
    dr, di = Q * (1 - sr), g * u * (1 - si)
    out.update(dx=g * np.sqrt(b2) * si, dr=dr, dlam=Q.sum(0) * sig(lam) / np.logaddexp(lam, 0), dh=carry, drb=dr.sum(0))
    if i is not None:
        out.update(di=di, dib=di.sum(0))
    if z is not None:
        sz = sig(z)
        slope = sz * (1 + z * (1 - sz))
        out["dz"] = a_(dy) * path[1:] * (np.abs(slope) + np.abs(z) / 4 if mag else slope)
    return out
