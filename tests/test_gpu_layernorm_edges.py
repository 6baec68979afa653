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
