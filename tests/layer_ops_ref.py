"""The layer operators in 64 bits, token by token, for one sequence (numpy), and the
tolerances of the comparisons.

Tolerances.  An output is rounded once to its type: half a step, eps / 2 relative (and half
the smallest subnormal).  Before that every value is a sum of products taken in 32 bits.  A
sum of n terms, each off by at most k roundings, is off by at most (n + k) 2^-24 times the
sum S of the terms' absolute values.  S is what these same functions give on absolute
values (``mag=True``).  The recurrences add the roundings of a step to those of the steps
before: a step is one exponential (2^-22 and the rounding of its argument, whose effect
|dt A| exp(-|dt A|) 2^-24 is below that), three products and sums, so (L + n + 64) 2^-22 S
covers L steps, sums over n terms and the functions (softplus, SiLU: a few 2^-23 each)."""
import numpy as np

EPS = {"fp32": 2.0 ** -23, "bf16": 2.0 ** -7, "fp16": 2.0 ** -10, "e4m3": 2.0 ** -3}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "e4m3": 2.0 ** -9}


def tol(ref, S, dtype, terms):
    return EPS[dtype] / 2 * np.abs(ref) * (1 + 2.0 ** -10) + TINY[dtype] / 2 + (terms + 64) * 2.0 ** -22 * S + 1e-37


def sigmoid(x):
    return 1 / (1 + np.exp(-x))


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    return sigmoid(x) * (1 + x * (1 - sigmoid(x)))


def norm(x, r, w, eps):
    h = x if r is None else x + r
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, y if w is None else y * w


def norm_back(h, w, dy, dh, eps, mag=False):
    rstd = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    a = np.abs if mag else (lambda v: v)
    hat, wdy = a(h * rstd), a(dy if w is None else dy * w)
    inner = hat * (wdy * hat).mean(-1, keepdims=True)
    dx = rstd * (wdy + inner if mag else wdy - inner)
    return dx if dh is None else dx + a(dh), (a(dy) * hat).sum(0)


def conv(x, w, b, act, state, mag=False):
    """x [L, C], w [C, W], state [W - 1, C] -> y, new state."""
    a = np.abs if mag else (lambda v: v)
    W, L = w.shape[1], x.shape[0]
    ext = np.concatenate([state, x])
    p = np.zeros_like(x) + (0 if b is None else a(b))
    for k in range(W):
        p = p + a(ext[k:k + L]) * a(w[:, k])
    return (p if mag or not act else silu(p)), ext[L:]


def conv_back(x, w, b, act, state, dy, dstate, mag=False):
    a = np.abs if mag else (lambda v: v)
    W, L = w.shape[1], x.shape[0]
    ext = np.concatenate([state, x])
    if act:
        p = np.zeros_like(x) + (0 if b is None else b)
        for k in range(W):
            p = p + ext[k:k + L] * w[:, k]
        if mag:  # SiLU' is at most 1.1 and off by at most |SiLU''| <= 1/2 times p's error
            pm, _ = conv(x, w, b, False, state, mag=True)
            dp = np.abs(dy) * (1.1 + 0.5 * pm)
        else:
            dp = dy * silu_slope(p)
    else:
        dp = a(dy)
    full = np.zeros_like(ext)
    dw = np.zeros(w.shape)
    for k in range(W):
        full[k:k + L] += dp * a(w[:, k])
        dw[:, k] = (dp * a(ext[k:k + L])).sum(0)
    if W > 1 and dstate is not None:
        full[L:] += a(dstate)
    return dict(dx=full[W - 1:], dw=dw, dbias=dp.sum(0), dstate=full[:W - 1])


def scan(x, dt, A, B, C, Dk, z, bias, softplus, h0, G, dy=None, dh=None, mag=False):
    """x, dt, z [L, D], B, C [L, G, N], h0 [D, N]; with dy the gradients too."""
    a = np.abs if mag else (lambda v: v)
    L, D = x.shape
    N = A.shape[1]
    raw = dt if bias is None else dt + bias
    step = np.logaddexp(raw, 0) if softplus else raw
    x, B, C, h = a(x), a(np.repeat(B, D // G, 1)), a(np.repeat(C, D // G, 1)), a(h0)
    gate = np.ones_like(x) if z is None else a(silu(z))
    dk = np.zeros(D) if Dk is None else a(Dk)
    ast = a(step)
    hs, e = [h], np.exp(step[:, :, None] * A)
    core = np.zeros_like(x)
    for t in range(L):
        h = e[t] * h + (ast[t] * x[t])[:, None] * B[t]
        hs.append(h)
        core[t] = (h * C[t]).sum(-1) + dk * x[t]
    out = dict(y=core * gate, h=h)
    if dy is None:
        return out
    dyg = a(dy) * gate
    slope = sigmoid(raw) if softplus else np.ones_like(raw)
    g = np.zeros((D, N)) if dh is None else a(dh)
    o = {k: np.zeros_like(x) for k in ("dx", "ddt")}
    dB, dC, dA = np.zeros((L, G, N)), np.zeros((L, G, N)), np.zeros((D, N))
    for t in reversed(range(L)):
        g = g + C[t] * dyg[t][:, None]
        dC[t] = (hs[t + 1] * dyg[t][:, None]).reshape(G, -1, N).sum(1)
        dB[t] = (g * (ast[t] * x[t])[:, None]).reshape(G, -1, N).sum(1)
        gB = (g * B[t]).sum(-1)
        q = g * e[t] * hs[t]
        dA += q * ast[t][:, None]
        o["ddt"][t] = ((q * a(A)).sum(-1) + gB * x[t]) * slope[t]
        o["dx"][t] = gB * ast[t] + dk * dyg[t]
        g = g * e[t]
    out.update(o, dB=dB, dC=dC, dA=dA, dD=(dyg * x).sum(0), ddt_bias=o["ddt"].sum(0), dh=g)
    if z is not None:
        s = silu_slope(z)
        out["dz"] = a(dy) * core * (np.abs(s) + np.abs(z) / 4 if mag else s)
    return out
