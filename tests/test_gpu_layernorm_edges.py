"""Layer norm on the GPU where kernels change hands: rows that a block of one warp walks.  References and tolerances
as in test_gpu_layernorm.py."""
import numpy as np
import pytest

import more_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_layer_ops import CODE, DT, _lib, close, dev, draw, host, rng, space, strided  # noqa: E402,F401
from test_gpu_layernorm import EPS, cfg_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", None), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("d,out,group", [(257, None, 0), (264, None, 0), (264, "e4m3", 100), (271, None, 0), (271, "e4m3", 0), (512, None, 0),
                                         (512, "e4m3", 128)])
def test_rows_that_one_warp_walks(d, out, group, dtype, r_dtype):
    """Rows of 257 to 512 channels, more than 1216 of them: each row's pieces are copied by other lanes than read them, and
    a block has no barrier but its warp's."""
    rows = 20000
    r = rng(70, d, group)
    x, xh = draw(r, (rows, d), dtype)
    res, rh = draw(r, (rows, d), r_dtype, 2.0) if r_dtype else (None, None)
    (w, wh), (b, bh) = draw(r, d, dtype), draw(r, d, dtype)
    cfg = cfg_of(rows, d, dtype, r_dtype, out_dtype=CODE[out or dtype], group=group)
    y = torch.empty(rows, d, device="cuda", dtype=DT[out or dtype])
    ro = torch.empty_like(res) if r_dtype else None
    scale = torch.empty(rows, -(-d // group) if group else 1, device="cuda") if out else None
    A.atlas_layernorm_forward(x, res, w, b, cfg, y, ro, scale)
    h, want, mag = R.layernorm(xh, rh, wh, bh, EPS)
    if r_dtype:
        close(ro, h, np.abs(xh) + np.abs(rh), r_dtype, 0, "residual")
    if out:
        g = group or d
        top = lambda v: np.stack([v[:, i:i + g].max(1) for i in range(0, d, g)], 1)  # noqa: E731
        close(host(scale) * 448, top(np.abs(want)), top(mag), "fp32", 0, "scale")
        step = np.repeat(host(scale), g, 1)[:, :d]
        close(host(y), want / step, mag / step, out, 0, "y")
    else:
        close(y, want, mag, dtype, 0, "y")


@pytest.mark.parametrize("rows,d,shift", [(5000, 24, 0), (5000, 37, 0), (4000, 128, 0), (40, 1000, 0), (1300, 512, 0), (1300, 1371, 0), (1300, 1371, 1),
                                          (1300, 2560, 0), (40, 8192, 0), (300, 9001, 0)])
@pytest.mark.parametrize("off,first", [(0.0, 1), (2.0, 1), (3.9, 1), (3.9, 8), (30.0, 8)])
def test_errors_in_32_bits_are_those_of_two_passes(rows, d, shift, off, first):
    """The rms error against 64 bits, whichever elements a row begins with (`first` of them, `off` deviations from the mean),
    is at most 1.5 times that of the mean first, then the deviations from it, in 32 bits."""
    r = rng(71, rows, d)
    x = strided(r, rows, d, "fp32", 0, shift)[0]
    x += 0.5 * dev(r.standard_normal((rows, 1)))
    x[:, :first] = x[:, first:].mean(1, keepdim=True) + off
    dy = draw(r, (rows, d), "fp32")[0]
    y, dx = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, device="cuda")
    cfg = cfg_of(rows, d, "fp32")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    A.atlas_layernorm_forward(x, None, None, None, cfg, y)
    h = x if shift == 0 else x.clone()
    A.atlas_layernorm_backward(h, None, dy, None, cfg, dx)

    def two_passes(x, dy):
        mid = x - x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(mid.square().mean(1, keepdim=True) + EPS)
        hat = mid * rstd
        return hat, rstd * (dy - dy.mean(1, keepdim=True) - hat * (dy * hat).mean(1, keepdim=True))
    exact, plain = two_passes(x.double(), dy.double()), two_passes(x, dy)
    for name, got, base, want in zip(("y", "dx"), (y, dx), plain, exact):
        rms = [float((v.double() - want).square().mean().sqrt()) for v in (got, base)]
        assert rms[0] <= 1.5 * rms[1], f"{name}: {rms[0]:.2e}, two passes {rms[1]:.2e}"
