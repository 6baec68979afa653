"""Layer norm on the GPU against the 64-bit reference of more_ops_ref.py: types, widths and alignments,
rows that start anywhere, 8-bit outputs, large means, rows that are not finite, gradients.  Tolerances:
see more_ops_ref.py."""
import os
import subprocess
import sys

import numpy as np
import pytest

import more_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_layer_ops import CODE, DT, _lib, close, dev, draw, host, rng, space, strided  # noqa: E402,F401

pytestmark = pytest.mark.gpu
EPS = 1e-5
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cfg_of(rows, d, dtype, r_dtype=None, **kw):
    return A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype or dtype], eps=EPS, **kw)


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,d,stride,shift", [
    (1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (9, 24, 0, 0), (33, 64, 72, 0), (300, 128, 0, 0), (9, 130, 0, 0), (4, 256, 0, 1),
    (5, 257, 0, 0), (7, 1000, 0, 0), (2, 1032, 0, 0), (6, 2048, 2064, 0), (3, 2050, 0, 0), (2, 8200, 0, 0), (1, 32768, 0, 0),
    (2, 32767, 0, 0), (5000, 24, 0, 0), (5000, 63, 0, 3), (1300, 264, 0, 0), (1300, 271, 0, 0), (1300, 1371, 1373, 5), (1250, 4104, 0, 0),
    (1240, 4099, 0, 1), (1230, 8191, 0, 0), (1220, 8192, 0, 0)])
def test_forward(rows, d, stride, shift, dtype, r_dtype):
    r = rng(40, rows, d)
    x, xh = strided(r, rows, d, dtype, stride, shift)
    res, rh = strided(r, rows, d, r_dtype, stride, shift, 2.0)
    (w, wh), (b, bh) = draw(r, d, dtype), draw(r, d, dtype)
    y, ro = strided(r, rows, d, dtype, stride, shift)[0], strided(r, rows, d, r_dtype, stride, shift)[0]
    ext = x.stride(0)
    cfg = cfg_of(rows, d, dtype, r_dtype, x_stride=ext, r_stride=ext, y_stride=ext)
    for residual, weight, bias, inplace in ((True, True, True, False), (True, False, True, True), (False, True, False, False)):
        h, want, mag = R.layernorm(xh, rh if residual else None, wh if weight else None, bh if bias else None, EPS)
        target = res if inplace else ro
        before = res.clone()
        A.atlas_layernorm_forward(x, res if residual else None, w if weight else None, b if bias else None, cfg, y,
                                  target if residual else None)
        close(y, want, mag, dtype, 0, "y")
        if residual:
            close(target, h, np.abs(xh) + np.abs(rh), r_dtype, 0, "residual")
        if inplace:
            res.copy_(before)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,d,stride", [(3, 7, 9), (2000, 37, 41), (1300, 271, 275), (1300, 1371, 1371), (40, 264, 272), (1300, 264, 280)])
def test_nothing_around_the_rows_is_used_or_written(rows, d, stride, dtype):
    """Rows in a storage of NaN: the gaps and what lies in front and behind stay, and enter nothing."""
    r = rng(41, rows, d)
    front = 3
    buf = torch.full((front + rows * stride + 5,), float("nan"), device="cuda").to(DT[dtype])
    out, res = buf.clone(), buf.clone()
    view = lambda t: t[front:front + (rows - 1) * stride + d].as_strided((rows, d), (stride, 1), front)  # noqa: E731
    x, xh = draw(r, (rows, d), dtype)
    view(buf).copy_(x)
    view(res).copy_(x)
    cfg = cfg_of(rows, d, dtype, x_stride=stride, r_stride=stride, y_stride=stride)
    A.atlas_layernorm_forward(view(buf), view(res), None, None, cfg, view(out), view(res))
    _, want, mag = R.layernorm(xh, xh, None, None, EPS)
    close(view(out), want, mag, dtype, 0, "y")
    g = buf.clone()
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    db = torch.empty(d, device="cuda")
    A.atlas_layernorm_backward(view(buf), None, view(buf), view(g), cfg, view(g), None, db)
    ref = R.layernorm_back(xh, None, xh, xh, EPS)
    close(view(g), *ref["dx"], dtype, 0, "dx")
    close(db, *ref["db"], "fp32", rows / 32, "db")
    for t in (buf, out, res, g):
        view(t).fill_(float("nan"))
        assert torch.isnan(t.float()).all()


@pytest.mark.parametrize("group", [0, 1, 5, 32, 100, 128, 4096])
@pytest.mark.parametrize("rows,d", [(3, 7), (40, 128), (5, 200), (3, 1024), (1400, 2048), (1400, 1371), (2, 4100), (1, 32768)])
def test_8_bits_are_the_32_bit_rows_rounded(rows, d, group):
    """q is y / scale to the nearest value, y the 32-bit output of the same rows."""
    r = rng(42, rows, d, group)
    x, res, w, b = (draw(r, s, "bf16")[0] for s in ((rows, d), (rows, d), d, d))
    y, q = torch.empty(rows, d, device="cuda"), torch.empty(rows, d, dtype=DT["e4m3"], device="cuda")
    g = group if 0 < group < d else d
    scale = torch.empty(rows, -(-d // g), device="cuda")
    A.atlas_layernorm_forward(x, res, w, b, cfg_of(rows, d, "bf16", out_dtype=A.F32), y)
    A.atlas_layernorm_forward(x, res, w, b, cfg_of(rows, d, "bf16", out_dtype=A.E4M3, group=group), q, None, scale)
    amax = torch.stack([p.abs().amax(1) for p in y.split(g, 1)], 1)
    assert torch.equal(scale, amax.clamp_min(1e-30) * (1 / 448))
    want = (y * (1 / scale).repeat_interleave(g, 1)[:, :d]).clamp(-448, 448).to(DT["e4m3"])
    assert torch.equal(q.float(), want.float()), int((q.float() != want.float()).sum())


@pytest.mark.parametrize("rows,d", [(5, 24), (5, 128), (5, 1000), (1300, 1371), (1300, 2048), (1240, 8192), (3, 20000)])
def test_a_large_mean_costs_nothing(rows, d):
    """Deviations of 1 about a mean of 4096, held exactly: no square of the mean and no rounded mean enters."""
    r = rng(43, rows, d)
    x, xh = draw(r, (rows, d), "fp32")
    x = x + 4096
    xh, dy = host(x), draw(r, (rows, d), "fp32")
    cfg = cfg_of(rows, d, "fp32")
    y = torch.empty_like(x)
    A.atlas_layernorm_forward(x, None, None, None, cfg, y)
    _, want, mag = R.layernorm(xh, None, None, None, EPS)
    close(y, want, mag, "fp32", 0, "y")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    w, wh = draw(r, d, "fp32")
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    cfg.w_dtype = A.F32
    A.atlas_layernorm_backward(x, w, dy[0], None, cfg, dx, dw)
    ref = R.layernorm_back(xh, wh, dy[1], None, EPS)
    close(dx, *ref["dx"], "fp32", 0, "dx")
    close(dw, *ref["dw"], "fp32", rows / 32, "dw")


@pytest.mark.parametrize("d", [7, 128, 1000, 1371, 8192, 20000])
def test_rows_that_are_equal_or_not_finite(d):
    """A row of equal numbers gives the bias; NaN and infinities stay in their row."""
    r = rng(44, d)
    rows = 6
    x, _ = draw(r, (rows, d), "fp32")
    (w, wh), (b, bh) = draw(r, d, "fp32"), draw(r, d, "fp32")
    x[1], x[2], x[4, d // 2], x[5, 0] = 0.0, 3.0, float("nan"), float("inf")
    cfg = cfg_of(rows, d, "fp32")
    y = torch.empty_like(x)
    A.atlas_layernorm_forward(x, None, w, b, cfg, y)
    for i in (1, 2):
        assert torch.equal(y[i], b)
    assert torch.isnan(y[4]).all() and torch.isnan(y[5]).any()
    for i in (0, 3):
        _, want, mag = R.layernorm(host(x[i:i + 1]), None, wh, bh, EPS)
        close(y[i:i + 1], want, mag, "fp32", 0, "y")
    dy, dx = torch.ones_like(x), torch.empty_like(x)
    A.atlas_layernorm_backward(x, w, dy, None, cfg, dx)
    assert torch.isfinite(dx[:4]).all() and torch.isnan(dx[4]).all()


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,d,stride,shift", [
    (0, 16, 0, 0), (1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (700, 64, 72, 0), (5000, 128, 0, 0), (9, 130, 0, 1), (7, 1000, 0, 0),
    (1000, 1032, 0, 0), (6, 2050, 0, 0), (700, 2560, 0, 0), (700, 1371, 1375, 3), (1500, 5000, 0, 0), (900, 3001, 0, 0),
    (500, 8192, 0, 0), (500, 8191, 0, 0), (2, 20000, 0, 0), (70, 8193, 8195, 1), (2, 32768, 0, 0)])
def test_backward(rows, d, stride, shift, dtype, r_dtype):
    r = rng(45, rows, d)
    h, hh = strided(r, rows, d, r_dtype, stride, shift, 2.0)
    dy, dyh = strided(r, rows, d, dtype, stride, shift)
    dh, dhh = strided(r, rows, d, r_dtype, stride, shift)
    w, wh = draw(r, d, dtype)
    ext = max(d, h.stride(0)) if rows else 0
    cfg = cfg_of(rows, d, dtype, r_dtype, r_stride=ext, y_stride=ext)
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    for up, weight, bias, inplace in ((True, True, True, False), (False, False, True, False), (True, True, False, True), (False, False, False, False)):
        dx = strided(r, rows, d, r_dtype, stride, shift)[0]
        dw, db = torch.full((d,), 9.0, device="cuda"), torch.full((d,), 9.0, device="cuda")
        if inplace:
            dx.copy_(dh)
        A.atlas_layernorm_backward(h, w if weight else None, dy, (dx if inplace else dh) if up else None, cfg, dx,
                                   dw if weight else None, db if bias else None)
        if rows:
            ref = R.layernorm_back(hh, wh if weight else None, dyh, dhh if up else None, EPS)
            close(dx, *ref["dx"], r_dtype, 0, "dx")
        else:
            ref = dict(dw=(np.zeros(d),) * 2, db=(np.zeros(d),) * 2)
        close(dw, *(ref["dw"] if weight else (np.full(d, 9.0), np.zeros(d))), "fp32", rows / 32, "dw")
        close(db, *(ref["db"] if bias else (np.full(d, 9.0), np.zeros(d))), "fp32", rows / 32, "db")


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "fp16"), ("fp16", "bf16")])
@pytest.mark.parametrize("rows,d", [(3, 24), (2000, 128), (5, 1032), (1300, 1032), (1300, 1371), (1300, 1370)])
def test_both_16_bit_types_at_once(rows, d, dtype, r_dtype):
    r = rng(49, rows, d)
    (x, xh), (res, rh), (w, wh) = draw(r, (rows, d), dtype), draw(r, (rows, d), r_dtype), draw(r, d, "fp16")
    cfg = cfg_of(rows, d, dtype, r_dtype, w_dtype=A.F16, out_dtype=A.F32)
    y, ro = torch.empty(rows, d, device="cuda"), torch.empty_like(res)
    A.atlas_layernorm_forward(x, res, w, w, cfg, y, ro)
    h, want, mag = R.layernorm(xh, rh, wh, wh, EPS)
    close(y, want, mag, "fp32", 0, "y")
    close(ro, h, np.abs(xh) + np.abs(rh), r_dtype, 0, "residual")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    dx, dw, db = torch.empty_like(res), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    A.atlas_layernorm_backward(res, w, x, res, cfg, dx, dw, db)
    ref = R.layernorm_back(rh, wh, xh, rh, EPS)
    close(dx, *ref["dx"], r_dtype, 0, "dx")
    close(dw, *ref["dw"], "fp32", rows / 32, "dw")
    close(db, *ref["db"], "fp32", rows / 32, "db")


@pytest.mark.parametrize("d", [1371, 1370, 1024])
@pytest.mark.parametrize("shifts", [(0, 0, 0), (1, 1, 1), (0, 1, 0), (1, 0, 1)])
def test_rows_that_begin_on_either_side_of_four_bytes(d, shifts):
    """Pairs where all tensors' rows begin alike, one by one where they do not; strides odd and even."""
    rows = 1400
    for stride in (d, d + 1):
        r = rng(50, d, stride)
        (x, xh), (res, rh) = (strided(r, rows, d, "bf16", stride, n) for n in shifts[:2])
        y = strided(r, rows, d, "bf16", stride, shifts[2])[0]
        cfg = cfg_of(rows, d, "bf16", x_stride=stride, r_stride=stride, y_stride=stride)
        A.atlas_layernorm_forward(x, res, None, None, cfg, y)
        _, want, mag = R.layernorm(xh, rh, None, None, EPS)
        close(y, want, mag, "bf16", 0, "y")
        space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
        db = torch.empty(d, device="cuda")
        A.atlas_layernorm_backward(res, None, x, None, cfg, y, None, db)
        ref = R.layernorm_back(rh, None, xh, None, EPS)
        close(y, *ref["dx"], "bf16", 0, "dx")
        close(db, *ref["db"], "fp32", rows / 32, "db")


def test_gradients_are_the_differences():
    """The kernels' gradients along a direction against differences of the kernels' own outputs, in 32 bits: the
    difference of the sums of rows * d products, each off by a few 2^-24, divided by a step of 2^-5."""
    rows, d, step = 12, 200, 2.0 ** -5
    r = rng(46)
    h, dy, w, b = (draw(r, s, "fp32")[0] for s in ((rows, d), (rows, d), d, d))
    cfg = cfg_of(rows, d, "fp32")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    dx, dw, db = torch.empty_like(h), torch.empty_like(w), torch.empty_like(b)
    A.atlas_layernorm_backward(h, w, dy, None, cfg, dx, dw, db)

    def loss(h, w, b):
        y = torch.empty_like(h)
        A.atlas_layernorm_forward(h, None, w, b, cfg, y)
        return float((y.double() * dy.double()).sum())
    for at, (v, g) in enumerate(((h, dx), (w, dw), (b, db))):
        u = draw(r, v.shape, "fp32")[0]
        u /= u.norm()  # a direction of length 1: the third derivative is a few times 1, the difference off by step^2 / 6 of it
        ends = []
        for sign in (1, -1):
            args = [h, w, b]
            args[at] = v + sign * step * u
            ends.append(loss(*args))
        want = float((g.double() * u.double()).sum())
        assert abs((ends[0] - ends[1]) / (2 * step) - want) < 1e-3 * (1 + float(g.norm()))


def test_rows_past_32_bits():
    """More than 2^32 elements: the last rows are as they are alone."""
    rows, d = (1 << 32) // 2048 + 3, 2048
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-5:] = dev(rng(47).standard_normal((5, d)), "bf16")
    y = torch.empty_like(x)
    A.atlas_layernorm_forward(x, None, None, None, cfg_of(rows, d, "bf16"), y)
    one = torch.empty(5, d, dtype=torch.bfloat16, device="cuda")
    A.atlas_layernorm_forward(x[-5:], None, None, None, cfg_of(5, d, "bf16"), one)
    assert (y[-5:].float() - one.float()).abs().max() <= 2.0 ** -7 * one.abs().max() and not y[:-5:997].any() and one.abs().max() > 1


@pytest.mark.parametrize("rows,d", [(5000, 128), (3000, 1371), (40, 9000)])
def test_captured_on_another_stream_with_equal_bits(rows, d):
    """Two captured calls with a workspace each, replayed together on two streams, give the eager call's bits."""
    r = rng(48, rows, d)
    h, dy, w = (draw(r, s, "bf16")[0] for s in ((rows, d), (rows, d), d))

    def plan():
        cfg = cfg_of(rows, d, "bf16")
        space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
        return cfg, torch.empty_like(h), torch.empty_like(h), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")

    def call(p):
        A.atlas_layernorm_forward(h, None, w, w, p[0], p[1])
        A.atlas_layernorm_backward(h, w, dy, dy, *p[:1], *p[2:])
    eager = plan()
    call(eager)
    graphs = []
    for _ in range(2):
        p, g, s = plan(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            call(p)
        graphs.append((p, g, s))
    torch.cuda.synchronize()
    for p, g, s in graphs:
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for p, _, _ in graphs:
        for got, want in zip(p[1:], eager[1:]):
            assert torch.equal(got, want)


def test_tensors_are_checked():
    x, w = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    cfg = cfg_of(4, 64, "bf16")
    space(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    f, n = torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")
    for bad in ((x.float(), None, w, w, x), (x, None, w.float(), w, x), (x, None, w, w.float(), x), (x, None, w, w[:32], x),
                (x[:3], None, w, w, x), (x, x[:3], w, w, x), (x, None, w, w, x[:2]), (x.cpu(), None, w, w, x)):
        with pytest.raises(A.AtlasError):
            A.atlas_layernorm_forward(*bad[:4], cfg, bad[4])
    for dw, db in ((n, f), (f, n), (f.bfloat16(), f), (f, f.cpu())):
        with pytest.raises(A.AtlasError):
            A.atlas_layernorm_backward(x, w, x, None, cfg, x.clone(), dw, db)


@pytest.mark.parametrize("rows,d", [(3, 128), (5, 200), (4, 2048), (1300, 1024), (1300, 1371), (3, 8200), (2, 32767)])
def test_deviations_whose_squares_leave_32_bits(rows, d):
    """A first element of 1e18: the squares of the distances to it do not add up in 32 bits, those of the distances to the mean
    do.  Where they do not either (1e25), the standard deviation is infinite: the row is its bias, and its dx is 0."""
    r = rng(51, rows, d)
    x, _ = draw(r, (rows, d), "fp32")
    x[0, 0], x[1, 0], x[-1, 0] = 1e18, 1e18, 1e25
    xh = host(x)
    (w, wh), (b, bh) = draw(r, d, "fp32"), draw(r, d, "fp32")
    (dy, dyh) = draw(r, (rows, d), "fp32")
    cfg = cfg_of(rows, d, "fp32")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    A.atlas_layernorm_forward(x, None, w, b, cfg, y)
    A.atlas_layernorm_backward(x, w, dy, None, cfg, dx)
    _, want, mag = R.layernorm(xh[:-1], None, wh, bh, EPS)
    # (an element's distance to the first one is rounded to that one's last place: 2^-24 |h_0 - mu| rstd <= 2^-24 sqrt(d))
    mag[:2] += np.sqrt(d) * np.abs(wh)
    close(y[:-1], want, mag, "fp32", 0, "y")
    assert torch.equal(y[-1], b) and not dx[-1].any()
    close(dx[2:-1], *[v[2:] for v in R.layernorm_back(xh[:-1], wh, dyh[:-1], None, EPS)["dx"]], "fp32", 0, "dx")
    assert torch.isfinite(dx).all()


def test_sums_do_not_depend_on_earlier_calls():
    """The blocks that share the rows are the same whatever ran before: dw's bits are those of a fresh process."""
    code = """if True:
        import sys, zlib, torch
        import test_memorization_recurrent_gb300 as A
        for d in map(int, sys.argv[1:]):
            torch.manual_seed(0)
            h, dy = torch.randn(3000, d, device="cuda"), torch.randn(3000, d, device="cuda")
            cfg = A.make_norm_cfg(3000, d, dtype=A.F32, r_dtype=A.F32, w_dtype=A.F32, out_dtype=A.F32)
            n = A.atlas_layernorm_backward_workspace_bytes(cfg)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            cfg.workspace, cfg.workspace_bytes, cfg.held = ws.data_ptr(), n, (ws,)
            dw, w = torch.empty(d, device="cuda"), torch.ones(d, device="cuda")
            A.atlas_layernorm_backward(h, w, dy, None, cfg, torch.empty_like(h), dw)
            print(d, zlib.crc32(dw.cpu().numpy().tobytes()))
    """
    runs = [subprocess.run([sys.executable, "-c", code, *order], capture_output=True, text=True, timeout=300, cwd=ROOT)
            for order in (("4200", "512"), ("512", "4200"))]
    for run in runs:
        assert run.returncode == 0, run.stderr
    first, second = (sorted(run.stdout.split("\n")) for run in runs)
    assert first == second
