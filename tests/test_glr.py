"""The gated linear recurrence without a GPU: refusals before any launch, sizes, and the gradients of the 64-bit
reference."""
import numpy as np
import pytest

import more_ops_ref as R
import test_memorization_recurrent_gb300 as A
from test_memorization_recurrent_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.load_library()


def forward(lib, cfg, x=16, r=16, i=16, z=None, lam=16, rb=None, ib=None, y=16, h0=None, h1=None, kept=None):
    return lib.atlas_glr_forward(x, r, i, z, lam, rb, ib, cfg, y, h0, h1, kept, None)


def backward(lib, cfg, x=16, r=16, i=16, z=None, lam=16, rb=None, ib=None, h0=None, kept=None, dy=16, dh=None, dx=16, dr=16,
             di=16, dz=None, dlam=16, drb=None, dib=None):
    return lib.atlas_glr_backward(x, r, i, z, lam, rb, ib, cfg, h0, kept, dy, dh, dx, dr, di, dz, dlam, drb, dib, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), A.ERR_INVALID), (dict(L=-1), A.ERR_INVALID), (dict(D=0), A.ERR_INVALID), (dict(dtype=A.E4M3), A.ERR_INVALID),
    (dict(dtype=-1), A.ERR_INVALID), (dict(c=0.0), A.ERR_INVALID), (dict(c=-1.0), A.ERR_INVALID), (dict(c=float("nan")), A.ERR_INVALID),
    (dict(c=float("inf")), A.ERR_INVALID), (dict(r_strides=(8, -8)), A.ERR_INVALID), (dict(y_strides=(-1, 8)), A.ERR_INVALID),
    (dict(slot=16, n_slots=0), A.ERR_INVALID), (dict(B=65536), A.ERR_UNSUPPORTED), (dict(B=60000, L=2 ** 31 - 1, D=4096), A.ERR_UNSUPPORTED),
    (dict(D=2 ** 31 - 1), A.ERR_UNSUPPORTED),
])
def test_descriptions_refused(lib, kw, code):
    cfg = A.make_glr_cfg(**{**dict(B=2, L=5, D=8), **kw})
    assert forward(lib, cfg) == code
    assert backward(lib, cfg) in (code, A.ERR_UNSUPPORTED)
    assert lib.atlas_glr_workspace_bytes(cfg) == lib.atlas_glr_kept_bytes(cfg) == lib.atlas_glr_backward_workspace_bytes(cfg) == 2 ** 64 - 1


def test_pointers_refused(lib):
    cfg = A.make_glr_cfg(2, 5, 8)
    for bad in (dict(x=None), dict(r=None), dict(lam=None), dict(y=None), dict(i=None, ib=16), dict(x=17), dict(r=17), dict(i=17),
                dict(z=17), dict(y=17), dict(lam=18), dict(rb=18), dict(ib=18), dict(h0=18), dict(h1=18), dict(kept=18)):
        assert forward(lib, cfg, **bad) == A.ERR_INVALID, bad
    for bad in (dict(x=None), dict(r=None), dict(lam=None), dict(dy=None), dict(dx=None), dict(dr=None), dict(dlam=None), dict(i=None),
                dict(di=None), dict(z=16), dict(dz=16), dict(rb=16), dict(drb=16), dict(ib=16), dict(dib=16), dict(i=None, di=None, ib=16, dib=16),
                dict(dy=17), dict(dx=17), dict(dr=17), dict(di=17), dict(dlam=18), dict(dh=18), dict(kept=18)):
        assert backward(lib, cfg, **bad) == A.ERR_INVALID, bad
    assert forward(lib, cfg) == backward(lib, cfg) == A.ERR_WORKSPACE
    assert backward(lib, A.make_glr_cfg(2, 5, 8, slot=16, n_slots=4)) == A.ERR_UNSUPPORTED
    assert lib.atlas_glr_forward(16, 16, 16, None, 16, None, None, None, 16, None, None, None, None) == A.ERR_INVALID
    assert forward(lib, A.make_glr_cfg(0, 5, 8), x=None, r=None, y=None) == A.OK
    for name in ("x", "r", "i"):
        assert backward(lib, A.make_glr_cfg(2, 5, 8, **{name + "_strides": (1, 2)})) == A.ERR_INVALID
    assert backward(lib, A.make_glr_cfg(2, 5, 8, z_strides=(40, 4)), z=16, dz=16) == A.ERR_INVALID
    assert forward(lib, A.make_glr_cfg(2, 5, 8, y_strides=(40, 4))) == A.ERR_INVALID


def test_sizes(lib):
    assert A.atlas_glr_workspace_bytes(A.make_glr_cfg(256, 1, 4096)) == 0   # single tokens
    assert A.atlas_glr_kept_bytes(A.make_glr_cfg(8, 4096, 2048)) == 256 * 2048 * 4
    need = A.atlas_glr_workspace_bytes(A.make_glr_cfg(1, 100000, 64))
    for ws, n in ((256, need - 1), (264, need), (None, need)):
        assert forward(lib, A.make_glr_cfg(1, 100000, 64, workspace=ws, workspace_bytes=n)) == A.ERR_WORKSPACE


@pytest.mark.parametrize("gated", [True, False])
def test_reference_gradient(gated):
    r = np.random.default_rng(5)
    L, D = 7, 4
    v = dict(x=r.standard_normal((L, D)), r=r.standard_normal((L, D)), i=r.standard_normal((L, D)) if gated else None,
             z=r.standard_normal((L, D)) if gated else None, lam=r.standard_normal(D) - 2, rb=r.standard_normal(D) * 0.1,
             ib=r.standard_normal(D) * 0.1 if gated else None, h0=r.standard_normal(D))
    dy, dh = r.standard_normal((L, D)), r.standard_normal(D)

    def run(grads=(), **kw):
        u = {**v, **kw}
        return R.glr(u["x"], u["r"], u["i"], u["z"], u["lam"], u["rb"], u["ib"], 3.0, u["h0"], *grads)

    def loss(**kw):
        o = run(**kw)
        return (o["y"] * dy).sum() + (o["h"] * dh).sum()
    g = run((dy, dh))
    for k, gk in dict(x="dx", r="dr", i="di", z="dz", lam="dlam", rb="drb", ib="dib", h0="dh").items():
        if v[k] is None:
            continue
        d = r.standard_normal(v[k].shape)
        step = (loss(**{k: v[k] + 1e-5 * d}) - loss(**{k: v[k] - 1e-5 * d})) / 2e-5
        assert abs(step - (g[gk] * d).sum()) < 1e-7, k


def test_size_of_the_kept_states_follows_the_description():
    """The binding works it out once, and again after a field that it depends on is set."""
    cfg = A.make_glr_cfg(2, 300, 40)
    cfg.kept_bytes = A.atlas_glr_kept_bytes(cfg)
    cfg.workspace_bytes = 5
    assert cfg.kept_bytes == 5 * 40 * 4  # one string: 600 rows
    cfg.L = 600
    assert cfg.kept_bytes is None and A.atlas_glr_kept_bytes(cfg) == 2 * 5 * 40 * 4
