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


@pytest.mark.parametrize("dtype,out", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,d,stride", [(9, 5, 0), (9, 24, 0), (40, 128, 0), (2000, 37, 0), (9, 1000, 0), (1300, 512, 0), (1300, 1371, 0), (1300, 1371, 1373),
                                           (1300, 2048, 0), (9, 8200, 0), (200, 9001, 0), (9, 20000, 0)])
def test_rows_next_to_the_largest_number(rows, d, stride, dtype, out):
    """The type's lowest value as first element, as first eight, everywhere, and in turn with its largest: neither the distances to
    a number nor their sums fit in 32 bits.  The variance does not either (or is 0): the row is its bias, its dx is dh, it adds
    nothing to dw, and the other rows are theirs."""
    r = rng(72, rows, d)
    x, _ = strided(r, rows, d, dtype, stride)
    low = float(torch.finfo(DT[dtype]).min)
    where = {1: slice(0, 1), 2: slice(0, 8), 4: slice(0, d), 6: slice(0, d, 2), 7: slice(d - 1, d)}
    for row, at in where.items():
        x[row, at] = low
    x[6, 1::2] = -low
    (w, _), (b, bh), (dy, dyh), (up, _) = draw(r, d, dtype), draw(r, d, dtype), draw(r, (rows, d), dtype), draw(r, (rows, d), dtype)
    y = torch.empty(rows, d, device="cuda", dtype=DT[out])
    cfg = cfg_of(rows, d, dtype, x_stride=stride, out_dtype=CODE[out])
    A.atlas_layernorm_forward(x, None, w, b, cfg, y)
    h, dx, dw, db = x.contiguous(), torch.empty_like(up), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    A.atlas_layernorm_backward(h, w, dy, up, cfg, dx, dw, db)
    bias = b.to(DT[out])
    for row in where:
        assert torch.equal(y[row], bias), row
        assert torch.equal(dx[row], up[row]), row
    others = [i for i in range(rows) if i not in where]
    _, want, mag = R.layernorm(host(h)[others], None, host(w), bh, EPS)
    close(y[others], want, mag, out, 0, "y")
    ref = R.layernorm_back(host(h)[others], host(w), dyh[others], host(up)[others], EPS)
    close(dx[others], *ref["dx"], dtype, 0, "dx")
    close(dw, *ref["dw"], "fp32", rows / 32, "dw")
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("d", [1, 2])
def test_more_rows_than_32_bits_count(d):
    """The last of 2^31 + 9 rows are as they are alone, forward and backward; dbias is of all."""
    rows, n = 2 ** 31 + 9, 300
    r = rng(73, d)
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-n:] = dev(r.standard_normal((n, d)), "bf16")
    b = dev(r.standard_normal(d), "bf16")
    y = torch.empty_like(x)
    A.atlas_layernorm_forward(x, None, None, b, cfg_of(rows, d, "bf16"), y)
    one = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    A.atlas_layernorm_forward(x[-n:], None, None, b, cfg_of(n, d, "bf16"), one)
    assert torch.equal(y[-n:], one) and bool((y[:-n:99991] == b).all())
    cfg = cfg_of(rows, d, "bf16")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    db = torch.empty(d, device="cuda")
    A.atlas_layernorm_backward(x, None, x, None, cfg, y, None, db)
    small = cfg_of(n, d, "bf16")
    space(small, A.atlas_layernorm_backward_workspace_bytes(small))
    A.atlas_layernorm_backward(x[-n:], None, x[-n:], None, small, one, None, None)
    # (one row a lane or several: other orders of a row's sums)
    assert (y[-n:].float() - one.float()).abs().max() <= 2.0 ** -6 * max(1.0, float(one.float().abs().max()))
    ref = host(x[-n:])
    close(db, ref.sum(0), np.abs(ref).sum(0), "fp32", n, "db")
