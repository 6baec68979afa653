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
