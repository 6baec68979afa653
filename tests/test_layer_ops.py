"""Layer operators without a GPU: the library exports what its header declares, bad
descriptions and pointers are refused before any launch, and the 64-bit references the GPU
tests compare with have the gradients that differences give."""
import ctypes
import os
import re

import numpy as np
import pytest

import layer_ops_ref as R
import test_memorization_recurrent_gb300 as A
from test_memorization_recurrent_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "atlas_ops.h")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.load_library()


def test_exports_are_the_header(lib):
    names = set(re.findall(r"^(?:int|size_t)\s+(atlas_\w+)\s*\(", open(HEADER).read(), flags=re.M))
    assert names == set(A.OPS_EXPORTS)
    for n in names:
        ctypes.cast(getattr(lib, n), ctypes.c_void_p)


# ------------------------------------------------------------------ norm

def norm_call(lib, cfg, x=16, r=None, w=None, y=16, ro=None, s=None):
    return lib.atlas_norm_forward(x, r, w, cfg, y, ro, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), A.ERR_INVALID), (dict(d=0), A.ERR_INVALID), (dict(group=-1), A.ERR_INVALID),
    (dict(dtype=A.E4M3), A.ERR_INVALID), (dict(r_dtype=3), A.ERR_INVALID), (dict(w_dtype=9), A.ERR_INVALID),
    (dict(out_dtype=4), A.ERR_INVALID), (dict(eps=-1.0), A.ERR_INVALID), (dict(eps=float("nan")), A.ERR_INVALID),
    (dict(x_stride=-8), A.ERR_INVALID), (dict(y_stride=7), A.ERR_INVALID), (dict(r_stride=3), A.ERR_INVALID),
    (dict(d=A.NORM_MAX_D + 1), A.ERR_UNSUPPORTED),
])
def test_norm_descriptions_refused(lib, kw, code):
    cfg = A.make_norm_cfg(**{**dict(rows=4, d=8), **kw})
    assert norm_call(lib, cfg) == code
    assert lib.atlas_norm_backward(16, 16, 16, None, cfg, 16, 16, None) == code
    assert lib.atlas_norm_backward_workspace_bytes(cfg) == 2 ** 64 - 1


def test_norm_pointers_refused(lib):
    cfg = A.make_norm_cfg(4, 8)
    assert norm_call(lib, cfg, x=None) == norm_call(lib, cfg, y=None) == A.ERR_INVALID
    assert norm_call(lib, cfg, s=16) == A.ERR_INVALID             # scales without 8 bits
    assert norm_call(lib, cfg, x=17) == A.ERR_INVALID             # not on an element
    q = A.make_norm_cfg(4, 8, out_dtype=A.E4M3)
    assert norm_call(lib, q) == A.ERR_INVALID                     # 8 bits without scales
    assert lib.atlas_norm_backward(16, None, 16, None, cfg, 16, 16, None) == A.ERR_INVALID
    assert lib.atlas_norm_backward(16, 16, 16, None, cfg, 16, 16, None) == A.ERR_WORKSPACE
    assert norm_call(lib, A.make_norm_cfg(0, 8), x=None, y=None) == A.OK


# ------------------------------------------------------------------ conv

def conv_call(lib, cfg, x=16, w=16, b=None, y=16, s0=None, s1=None):
    return lib.atlas_conv_forward(x, w, b, cfg, y, s0, s1, None)


def conv_back(lib, cfg, dw=16, ws=None):
    return lib.atlas_conv_backward(16, 16, None, cfg, None, 16, None, 16, dw, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), A.ERR_INVALID), (dict(L=-1), A.ERR_INVALID), (dict(C=0), A.ERR_INVALID),
    (dict(W=0), A.ERR_INVALID), (dict(W=A.CONV_MAX_W + 1), A.ERR_UNSUPPORTED), (dict(act=2), A.ERR_INVALID),
    (dict(dtype=A.E4M3), A.ERR_INVALID), (dict(w_dtype=7), A.ERR_INVALID), (dict(head_dim=3), A.ERR_INVALID),
    (dict(head_dim=-4), A.ERR_INVALID), (dict(x_strides=(-1, 8)), A.ERR_INVALID),
    (dict(slot=16, n_slots=0), A.ERR_INVALID),
])
def test_conv_descriptions_refused(lib, kw, code):
    cfg = A.make_conv_cfg(**{**dict(B=2, L=5, C=8, W=4), **kw})
    assert conv_call(lib, cfg) == code
    assert conv_back(lib, cfg) in (code, A.ERR_UNSUPPORTED)
    assert lib.atlas_conv_backward_workspace_bytes(cfg) == 2 ** 64 - 1


@pytest.mark.parametrize("strides", [(40, 4), (4, 8), (16, 0), (0, 8)])
def test_conv_overlapping_rows_refused(lib, strides):
    """Rows that are written must lie apart: y in the forward, dx in the backward."""
    assert conv_call(lib, A.make_conv_cfg(2, 5, 8, 4, y_strides=strides)) == A.ERR_INVALID
    assert conv_back(lib, A.make_conv_cfg(2, 5, 8, 4, x_strides=strides)) == A.ERR_INVALID


def test_conv_overlapping_heads_refused(lib):
    assert conv_call(lib, A.make_conv_cfg(2, 5, 8, 4, head_dim=4, y_strides=(40, 4, 8))) == A.ERR_INVALID
    assert conv_call(lib, A.make_conv_cfg(2, 5, 8, 4, head_dim=4, y_strides=(30, 4, 20))) == A.ERR_INVALID


def test_conv_pointers_refused(lib):
    cfg = A.make_conv_cfg(2, 5, 8, 4)
    for bad in (dict(x=None), dict(y=None), dict(w=None), dict(x=17), dict(s0=17), dict(s1=1)):
        assert conv_call(lib, cfg, **bad) == A.ERR_INVALID
    assert conv_back(lib, cfg, dw=None) == A.ERR_INVALID
    assert conv_back(lib, cfg) == A.ERR_WORKSPACE
    assert conv_back(lib, A.make_conv_cfg(2, 5, 8, 4, slot=16, n_slots=4)) == A.ERR_UNSUPPORTED
    assert conv_call(lib, A.make_conv_cfg(0, 5, 8, 4), x=None, y=None, w=None) == A.OK


# ------------------------------------------------------------------ scan

def scan_call(lib, cfg, x=16, a=16, y=16, b=16):
    return lib.atlas_scan_forward(x, 16, a, b, 16, None, None, None, cfg, y, None, None, None)


def scan_back(lib, cfg, D=None, dD=None, z=None, dz=None, bias=None, dbias=None, dA=16, dx=16):
    return lib.atlas_scan_backward(16, 16, 16, 16, 16, D, z, bias, cfg, None, 16, None, dx, 16, dA, 16, 16,
                                   dD, dz, dbias, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), A.ERR_INVALID), (dict(L=-1), A.ERR_INVALID), (dict(D=0), A.ERR_INVALID), (dict(N=0), A.ERR_INVALID),
    (dict(G=3), A.ERR_INVALID), (dict(G=0), A.ERR_INVALID), (dict(N=A.SCAN_MAX_N + 1), A.ERR_UNSUPPORTED),
    (dict(B=65536), A.ERR_UNSUPPORTED), (dict(dtype=A.E4M3), A.ERR_INVALID), (dict(dt_strides=(8, -8)), A.ERR_INVALID),
    (dict(slot=16, n_slots=-1), A.ERR_INVALID),
])
def test_scan_descriptions_refused(lib, kw, code):
    cfg = A.make_scan_cfg(**{**dict(B=2, L=5, D=8, N=4), **kw})
    assert scan_call(lib, cfg) == code
    assert scan_back(lib, cfg) in (code, A.ERR_UNSUPPORTED)
    assert lib.atlas_scan_workspace_bytes(cfg) == lib.atlas_scan_backward_workspace_bytes(cfg) == 2 ** 64 - 1


def test_scan_pointers_refused(lib):
    cfg = A.make_scan_cfg(2, 5, 8, 4)
    for bad in (dict(x=None), dict(y=None), dict(a=None), dict(b=None), dict(x=17), dict(a=18)):
        assert scan_call(lib, cfg, **bad) == A.ERR_INVALID
    for bad in (dict(D=16), dict(dD=16), dict(z=16), dict(dz=16), dict(bias=16), dict(dbias=16), dict(dA=None), dict(dx=None)):
        assert scan_back(lib, cfg, **bad) == A.ERR_INVALID
    assert scan_back(lib, cfg) == A.ERR_WORKSPACE
    assert scan_back(lib, A.make_scan_cfg(2, 5, 8, 4, slot=16, n_slots=4)) == A.ERR_UNSUPPORTED
    # rows that are written lie apart: y, and in the backward the gradients with their inputs' strides
    assert scan_call(lib, A.make_scan_cfg(2, 5, 8, 4, y_strides=(40, 4))) == A.ERR_INVALID
    for name in ("x", "dt", "B", "C"):
        assert scan_back(lib, A.make_scan_cfg(2, 5, 8, 4, **{name + "_strides": (1, 2)})) == A.ERR_INVALID
    long = A.make_scan_cfg(1, 100000, 64, 16)
    assert lib.atlas_scan_workspace_bytes(long) > 0 and scan_call(lib, long) == A.ERR_WORKSPACE


def test_single_tokens_need_no_workspace(lib):
    assert A.atlas_scan_workspace_bytes(A.make_scan_cfg(256, 1, 4096, 16)) == 0


# ---------------------------------------------------- the references' gradients

def differences(f, x, d):
    """Directional derivative of f at x along d."""
    return (f(x + 1e-5 * d) - f(x - 1e-5 * d)) / 2e-5


def test_reference_norm_gradient():
    r = np.random.default_rng(0)
    h, w, dy, dh = r.standard_normal((3, 7)), r.standard_normal(7), r.standard_normal((3, 7)), r.standard_normal((3, 7))
    dx, dw = R.norm_back(h, w, dy, dh, 1e-6)
    d, dd = r.standard_normal((3, 7)), r.standard_normal(7)
    f = lambda h, w: (R.norm(h, None, w, 1e-6)[1] * dy).sum() + (h * dh).sum()  # noqa: E731
    assert abs(differences(lambda v: f(v, w), h, d) - (dx * d).sum()) < 1e-7
    assert abs(differences(lambda v: f(h, v), w, dd) - (dw * dd).sum()) < 1e-7


@pytest.mark.parametrize("W,L,act", [(1, 4, True), (4, 2, True), (4, 9, True), (3, 5, False), (4, 0, True)])
def test_reference_conv_gradient(W, L, act):
    r = np.random.default_rng(1)
    v = dict(x=r.standard_normal((L, 3)), w=r.standard_normal((3, W)), b=r.standard_normal(3), state=r.standard_normal((W - 1, 3)))
    dy, ds = r.standard_normal((L, 3)), r.standard_normal((W - 1, 3))
    g = R.conv_back(v["x"], v["w"], v["b"], act, v["state"], dy, ds)

    def loss(**kw):
        u = {**v, **kw}
        y, s = R.conv(u["x"], u["w"], u["b"], act, u["state"])
        return (y * dy).sum() + (s * ds).sum()
    for k, gk in (("x", "dx"), ("w", "dw"), ("b", "dbias"), ("state", "dstate")):
        d = r.standard_normal(v[k].shape)
        assert abs(differences(lambda u: loss(**{k: u}), v[k], d) - (g[gk] * d).sum()) < 1e-7, k


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_reference_scan_gradient(softplus, gate):
    r = np.random.default_rng(2)
    L, D, N, G = 6, 4, 3, 2
    v = dict(x=r.standard_normal((L, D)), dt=r.uniform(0.1, 1, (L, D)), A=-r.uniform(0.2, 2, (D, N)),
             B=r.standard_normal((L, G, N)), C=r.standard_normal((L, G, N)), Dk=r.standard_normal(D),
             z=r.standard_normal((L, D)) if gate else None, bias=r.standard_normal(D) * 0.1, h0=r.standard_normal((D, N)))
    dy, dh = r.standard_normal((L, D)), r.standard_normal((D, N))

    def run(grad=False, **kw):
        u = {**v, **kw}
        return R.scan(u["x"], u["dt"], u["A"], u["B"], u["C"], u["Dk"], u["z"], u["bias"], softplus, u["h0"], G,
                      *((dy, dh) if grad else ()))
    g = run(True)

    def loss(**kw):
        o = run(**kw)
        return (o["y"] * dy).sum() + (o["h"] * dh).sum()
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", Dk="dD", bias="ddt_bias", h0="dh")
    if gate:
        names["z"] = "dz"
    for k, gk in names.items():
        d = r.standard_normal(v[k].shape)
        assert abs(differences(lambda u: loss(**{k: u}), v[k], d) - (g[gk] * d).sum()) < 1e-7, k
