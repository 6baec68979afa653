"""Layer norm without a GPU: refusals before any launch, and the gradients of the 64-bit reference."""
import numpy as np
import pytest

import more_ops_ref as R
import test_memorization_recurrent_gb300 as A
from test_memorization_recurrent_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.load_library()


def forward(lib, cfg, x=16, r=None, w=None, b=None, y=16, ro=None, s=None):
    return lib.atlas_layernorm_forward(x, r, w, b, cfg, y, ro, s, None)


def backward(lib, cfg, h=16, w=16, dy=16, dh=None, dx=16, dw=None, db=None):
    return lib.atlas_layernorm_backward(h, w, dy, dh, cfg, dx, dw, db, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), A.ERR_INVALID), (dict(d=0), A.ERR_INVALID), (dict(group=-1), A.ERR_INVALID),
    (dict(dtype=A.E4M3), A.ERR_INVALID), (dict(r_dtype=3), A.ERR_INVALID), (dict(w_dtype=9), A.ERR_INVALID),
    (dict(out_dtype=4), A.ERR_INVALID), (dict(eps=0.0), A.ERR_INVALID), (dict(eps=-1.0), A.ERR_INVALID),
    (dict(eps=float("nan")), A.ERR_INVALID), (dict(eps=float("inf")), A.ERR_INVALID), (dict(x_stride=-8), A.ERR_INVALID),
    (dict(y_stride=7), A.ERR_INVALID), (dict(r_stride=3), A.ERR_INVALID), (dict(d=A.NORM_MAX_D + 1), A.ERR_UNSUPPORTED),
])
def test_descriptions_refused(lib, kw, code):
    cfg = A.make_norm_cfg(**{**dict(rows=4, d=8), **kw})
    assert forward(lib, cfg) == code
    assert backward(lib, cfg) == code
    assert lib.atlas_layernorm_backward_workspace_bytes(cfg) == 2 ** 64 - 1
    with pytest.raises(A.AtlasError):
        A.atlas_layernorm_backward_workspace_bytes(cfg)


def test_pointers_refused(lib):
    cfg = A.make_norm_cfg(4, 8, r_dtype=A.F32)
    for bad in (dict(x=None), dict(y=None), dict(s=16), dict(x=17), dict(y=17), dict(r=18), dict(ro=18), dict(w=17), dict(b=17)):
        assert forward(lib, cfg, **bad) == A.ERR_INVALID, bad
    assert forward(lib, A.make_norm_cfg(4, 8, out_dtype=A.E4M3)) == A.ERR_INVALID      # 8 bits without scales
    assert forward(lib, A.make_norm_cfg(4, 8, out_dtype=A.E4M3), s=18) == A.ERR_INVALID
    for bad in (dict(h=None), dict(dy=None), dict(dx=None), dict(h=18), dict(dy=17), dict(dh=18), dict(dx=18), dict(w=17),
                dict(dw=18), dict(db=18), dict(w=None, dw=16)):
        assert backward(lib, cfg, **bad) == A.ERR_INVALID, bad
    assert backward(lib, cfg, dw=16) == backward(lib, cfg, db=16) == backward(lib, cfg, w=None, db=16) == A.ERR_WORKSPACE
    assert lib.atlas_layernorm_forward(16, None, None, None, None, 16, None, None, None) == A.ERR_INVALID
    empty = A.make_norm_cfg(0, 8)
    assert forward(lib, empty, x=None, y=None) == A.OK
    assert backward(lib, empty, h=None, dy=None, dx=None) == A.OK


def test_short_workspaces_refused(lib):
    for rows, d in ((4, 8), (5, 20000), (100000, 128)):
        need = A.atlas_layernorm_backward_workspace_bytes(A.make_norm_cfg(rows, d))
        assert need > 0
        for ws, n in ((256, need - 1), (264, need), (None, need)):
            assert backward(lib, A.make_norm_cfg(rows, d, workspace=ws, workspace_bytes=n), dw=16) == A.ERR_WORKSPACE


def test_workspace_does_not_go_by_the_rows():
    """Partial sums are the blocks', not the rows' (but for two numbers a row beyond 8192 channels)."""
    small, large = (A.atlas_layernorm_backward_workspace_bytes(A.make_norm_cfg(n, 1024)) for n in (10 ** 5, 10 ** 7))
    assert small == large < 16 << 20


def test_reference_gradient():
    r = np.random.default_rng(0)
    h, dy, dh, w, b = (r.standard_normal(s) for s in ((3, 7), (3, 7), (3, 7), 7, 7))
    g = R.layernorm_back(h, w, dy, dh, 1e-5)
    f = lambda h, w, b: (R.layernorm(h, None, w, b, 1e-5)[1] * dy).sum() + (h * dh).sum()  # noqa: E731
    for at, (k, v) in enumerate((("dx", h), ("dw", w), ("db", b))):
        d = r.standard_normal(v.shape)
        plus, minus = [h, w, b], [h, w, b]
        plus[at], minus[at] = v + 1e-5 * d, v - 1e-5 * d
        assert abs((f(*plus) - f(*minus)) / 2e-5 - (g[k][0] * d).sum()) < 1e-7, k
