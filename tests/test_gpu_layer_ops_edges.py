"""Layer operators where they are easily wrong: 8-bit outputs beside 32-bit ones, norms without
eps, rows past the last, states that are not finite, starts that fall, layouts whose
dimensions lie in any order, batches of many sequences.  References and tolerances as in
test_gpu_layer_ops.py."""
import numpy as np
import pytest

import layer_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_layer_ops import CODE, DT, TYPES, Conv, Scan, _lib, close, dev, draw, host, rng, run_scan, space, status  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,d,group", [(8, 2048, 0), (3000, 2048, 128), (20000, 128, 32), (900, 1371, 100), (1300, 8200, 0)])
def test_8_bits_are_the_32_bit_rows_rounded(rows, d, group):
    """q is y / scale to the nearest value, y the 32-bit output of the same rows: the quotient, taken as
    y times the rounded 1 / scale, in 32 bits and no other steps."""
    r = rng(30, rows, d)
    x, res, w = (draw(r, s, "bf16")[0] for s in ((rows, d), (rows, d), (d,)))
    y, q = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, dtype=DT["e4m3"], device="cuda")
    g = group or d
    scale = torch.empty(rows, -(-d // g), device="cuda")
    A.atlas_norm_forward(x, res, w, A.make_norm_cfg(rows, d, out_dtype=A.F32), y)
    A.atlas_norm_forward(x, res, w, A.make_norm_cfg(rows, d, out_dtype=A.E4M3, group=group), q, None, scale)
    amax = torch.stack([p.abs().amax(1) for p in y.split(g, 1)], 1)
    assert torch.equal(scale, amax.clamp_min(1e-30) * (1 / 448))
    want = (y * (1 / scale).repeat_interleave(g, 1)[:, :d]).clamp(-448, 448).to(DT["e4m3"])
    assert torch.equal(q.float(), want.float()), int((q.float() != want.float()).sum())


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows", [1, 5, 9, 701])
@pytest.mark.parametrize("d", [64, 128, 256, 130, 520])
def test_norm_backward_without_eps(d, rows, dtype, r_dtype):
    """Rows that do not fill their block's places, eps = 0: dw is the sum over the rows there are."""
    r = rng(31, rows, d)
    h, hh = draw(r, (rows, d), r_dtype, 2.0)
    dy, dyh = draw(r, (rows, d), dtype)
    w, wh = draw(r, d, dtype)
    cfg = A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype], eps=0.0)
    space(cfg, A.atlas_norm_backward_workspace_bytes(cfg))
    dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
    A.atlas_norm_backward(h, w, dy, None, cfg, dx, dw)
    want, mag = (R.norm_back(hh, wh, dyh, None, 0.0, mag=m) for m in (False, True))
    close(dx, want[0], mag[0], r_dtype, 0, "dx")
    close(dw, want[1], mag[1], "fp32", rows / 32, "dw")


