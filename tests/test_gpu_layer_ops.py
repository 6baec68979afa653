"""Layer operators (norm, short convolution, selective scan) on the GPU against the 64-bit
references of layer_ops_ref.py: types, odd widths, lengths from none to several segments,
strides and alignment, packed sequences with empty ones and rows behind the last, state
slots with padding, streams and captured graphs, and a layer of them around the memory
update.  Tolerances: see layer_ops_ref.py."""
import numpy as np
import pytest

import layer_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402

pytestmark = pytest.mark.gpu
CODE = {"fp32": A.F32, "bf16": A.BF16, "fp16": A.F16, "e4m3": A.E4M3}
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
TYPES = ["fp32", "bf16", "fp16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from test_memorization_recurrent_gb300 import build
    build.build()


def rng(*key):
    return np.random.default_rng([7, *key])


def dev(a, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(DT[dtype])


def host(t):
    return t.double().cpu().numpy()


def draw(r, shape, dtype, scale=1.0):
    """A device tensor of a type and the values it holds, in 64 bits."""
    t = dev(r.standard_normal(shape) * scale, dtype)
    return t, host(t)


def close(got, ref, S, dtype, terms, what=""):
    got = host(got) if torch.is_tensor(got) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.size == 0:
        return
    over = np.abs(got - ref) - R.tol(ref, S, dtype, terms)
    assert np.isfinite(got).all() and (over <= 0).all(), f"{what}: off by {over.max():.3e} more than allowed"


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def space(cfg, nbytes):
    ws = torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")
    cfg.workspace, cfg.workspace_bytes = ws.data_ptr(), nbytes
    cfg.held = (cfg.held, ws)  # lives as long as its description


# ------------------------------------------------------------------ norm

def strided(r, rows, d, dtype, stride=0, shift=0, scale=1.0):
    """A [rows, d] view with a row stride, starting `shift` elements into its storage."""
    stride = stride or d
    t, _ = draw(r, rows * stride + shift + 8, dtype, scale)
    v = t[shift:shift + rows * stride].view(rows, stride)[:, :d]
    return v, host(v)


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,d,stride,shift", [
    (1, 1, 0, 0), (3, 7, 0, 0), (5, 16, 0, 0), (33, 64, 72, 0), (300, 128, 0, 0), (9, 130, 0, 0), (4, 256, 0, 1),
    (7, 1000, 0, 0), (2, 1032, 0, 0), (6, 2048, 2064, 0), (3, 2050, 0, 0), (2, 8200, 0, 0), (1, 32768, 0, 0), (2, 32767, 0, 0)])
def test_norm(rows, d, stride, shift, dtype, r_dtype):
    r = rng(1, rows, d)
    x, xh = strided(r, rows, d, dtype, stride, shift)
    res, rh = strided(r, rows, d, r_dtype, stride, shift, 2.0)
    w, wh = draw(r, d, dtype)
    y, ro = strided(r, rows, d, dtype, stride, shift)[0], strided(r, rows, d, r_dtype, stride, shift)[0]
    ext = x.stride(0)
    for residual, weight, inplace in ((True, True, False), (True, False, True), (False, True, False)):
        cfg = A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype], x_stride=ext, r_stride=ext, y_stride=ext)
        h, want = R.norm(xh, rh if residual else None, wh if weight else None, cfg.eps)
        target = res if inplace else ro
        before = res.clone()
        A.atlas_norm_forward(x, res if residual else None, w if weight else None, cfg, y, target if residual else None)
        close(y, want, np.abs(want), dtype, 0, "y")
        if residual:
            close(target, h, np.abs(xh) + np.abs(rh), r_dtype, 0, "residual")
        if inplace:
            res.copy_(before)


@pytest.mark.parametrize("group", [0, 1, 5, 32, 100, 128, 4096])
@pytest.mark.parametrize("rows,d", [(3, 7), (40, 128), (5, 200), (3, 1024), (4, 2048), (2, 4100)])
def test_norm_in_8_bits(rows, d, group):
    """q within half a step of y / scale; the scale to 32-bit precision; a row of zeros gives zeros."""
    r = rng(2, rows, d, group)
    x, xh = draw(r, (rows, d), "bf16")
    x[0], xh[0] = 0, 0
    w, wh = draw(r, d, "bf16")
    g = group if 0 < group < d else d
    n = -(-d // g)
    y = torch.empty(rows, d, dtype=DT["e4m3"], device="cuda")
    scale = torch.empty(rows, n, device="cuda")
    A.atlas_norm_forward(x, None, w, A.make_norm_cfg(rows, d, out_dtype=A.E4M3, group=group), y, None, scale)
    _, want = R.norm(xh, None, wh, 1e-6)
    amax = np.stack([np.abs(want[:, i:i + g]).max(1) for i in range(0, d, g)], 1)
    ref = np.maximum(amax, 1e-30) / 448
    assert (np.abs(host(scale) - ref) <= 2.0 ** -18 * ref).all()
    q = want / np.repeat(ref, g, 1)[:, :d]
    close(y, q, np.abs(q), "e4m3", 0, "q")
    assert (host(y)[0] == 0).all()
    assert np.abs(host(y)).max() == 448


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,d,stride,shift", [(0, 16, 0, 0), (1, 1, 0, 0), (3, 7, 0, 0), (700, 64, 72, 0), (5000, 128, 0, 0), (9, 130, 0, 1),
                                                 (7, 1000, 0, 0), (1000, 1032, 0, 0), (6, 2050, 0, 0), (700, 2560, 0, 0), (1500, 5000, 0, 0), (900, 3000, 0, 0), (2, 20000, 0, 0), (2, 32767, 0, 0)])
def test_norm_backward(rows, d, stride, shift, dtype, r_dtype):
    r = rng(3, rows, d)
    h, hh = strided(r, rows, d, r_dtype, stride, shift, 2.0)
    dy, dyh = strided(r, rows, d, dtype, stride, shift)
    dh, dhh = strided(r, rows, d, r_dtype, stride, shift)
    w, wh = draw(r, d, dtype)
    ext = max(d, h.stride(0)) if rows else 0
    for up, weight in ((True, True), (False, False)):
        cfg = A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype], r_stride=ext, y_stride=ext)
        space(cfg, A.atlas_norm_backward_workspace_bytes(cfg))
        dx, dw = strided(r, rows, d, r_dtype, stride, shift)[0], torch.full((d,), 9.0, device="cuda")
        args = (hh, wh if weight else None, dyh, dhh if up else None, cfg.eps)
        A.atlas_norm_backward(h, w if weight else None, dy, dh if up else None, cfg, dx, dw if weight else None)
        if rows:
            want, mag = R.norm_back(*args), R.norm_back(*args, mag=True)
            close(dx, want[0], mag[0], r_dtype, 0, "dx")
        else:
            want = mag = (None, np.zeros(d))
        if weight:
            close(dw, want[1], mag[1], "fp32", rows / 32, "dw")


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,d,group", [(1300, 264, 0), (2600, 2048, 128), (1250, 4104, 0), (1230, 8200, 256), (1220, 17000, 64)])
def test_norm_many_long_rows(rows, d, group, dtype, r_dtype):
    """Rows enough for blocks that walk several, one to eight vectors a thread; in place, and with an
    8-bit output too."""
    r = rng(24, rows, d)
    x, xh = draw(r, (rows, d), dtype)
    res, rh = draw(r, (rows, d), r_dtype, 2.0)
    w, wh = draw(r, d, dtype)
    h, want = R.norm(xh, rh, wh, 1e-6)
    keep, y = res.clone(), torch.empty_like(x)
    A.atlas_norm_forward(x, res, w, A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype]), y, res)
    close(y, want, np.abs(want), dtype, 0, "y")
    close(res, h, np.abs(xh) + np.abs(rh), r_dtype, 0, "residual")
    g = group or d
    q, scale = torch.empty(rows, d, dtype=DT["e4m3"], device="cuda"), torch.empty(rows, -(-d // g), device="cuda")
    A.atlas_norm_forward(x, keep, w, A.make_norm_cfg(rows, d, dtype=CODE[dtype], r_dtype=CODE[r_dtype], out_dtype=A.E4M3, group=group), q, None, scale)
    ref = np.maximum(np.stack([np.abs(want[:, i:i + g]).max(1) for i in range(0, d, g)], 1), 1e-30) / 448
    assert (np.abs(host(scale) - ref) <= 2.0 ** -18 * ref).all()
    v = want / np.repeat(ref, g, 1)[:, :d]
    close(q, v, np.abs(v), "e4m3", 0, "q")


def test_norm_rows_past_32_bits():
    """More than 2^32 elements: the last rows are as they are alone."""
    rows, d = (1 << 32) // 2048 + 3, 2048
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-5:] = dev(rng(4).standard_normal((5, d)), "bf16")
    y = torch.empty_like(x)
    A.atlas_norm_forward(x, None, None, A.make_norm_cfg(rows, d), y)
    one = torch.empty(5, d, dtype=torch.bfloat16, device="cuda")
    A.atlas_norm_forward(x[-5:], None, None, A.make_norm_cfg(5, d), one)
    assert torch.equal(y[-5:], one) and not y[:-5:997].any() and one.abs().max() > 1


# ------------------------------------------------------------------ sequences

LENS = [[5], [1, 1, 1], [0, 9, 0, 64, 3, 0], [40, 2, 0, 131], [700, 0, 333, 1]]


def packed(lens, behind=3, front=0):
    start = np.concatenate([[0], np.cumsum(lens)]) + front
    return torch.tensor(start, dtype=torch.int32, device="cuda"), int(start[-1]) + behind, start


# ------------------------------------------------------------------ conv

class Conv:
    """One call's data on both sides."""

    def __init__(self, r, B, L, C, W, dtype, act=True, bias=True, n=None, packed_rows=None):
        lead = (packed_rows,) if packed_rows else (B, L)
        self.x, self.xh = draw(r, (*lead, C), dtype)
        self.w, self.wh = draw(r, (C, W), dtype, W ** -0.5)
        self.b, self.bh = draw(r, C, dtype, 0.2) if bias else (None, None)
        self.s, self.sh = draw(r, (n or B, W - 1, C), dtype)
        self.dy, self.dyh = draw(r, (*lead, C), dtype)
        self.ds, self.dsh = draw(r, (B, W - 1, C), "fp32")
        self.act = act

    def check(self, y, new, rows, state, dtype, what):
        x = self.xh[rows]
        want, ws = R.conv(x, self.wh, self.bh, self.act, state)
        S, _ = R.conv(x, self.wh, self.bh, self.act, state, mag=True)
        close(y, want, 1.1 * S, dtype, 0, what)  # |SiLU'| <= 1.1
        assert new is None or (host(new) == ws).all(), what


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,C,W,shift", [(2, 5, 8, 4, 0), (1, 1, 3, 4, 0), (3, 1, 64, 4, 0), (2, 2, 40, 4, 0), (1, 65, 264, 1, 0), (2, 64, 48, 2, 0),
                                           (2, 300, 33, 3, 0), (1, 200, 256, 5, 1), (2, 9, 16, 8, 0), (1, 7, 16, 8, 0), (2, 130, 520, 8, 0), (2, 0, 8, 4, 0)])
def test_conv(B, L, C, W, shift, dtype):
    r = rng(5, B, L, C, W)
    d = Conv(r, B, L, C, W, dtype, act=W != 5, bias=C != 48)
    if shift:  # off the 16-byte grid
        d.x = torch.cat([d.x.new_zeros(shift), d.x.flatten()])[shift:].view(B, L, C)
    y, new = torch.zeros_like(d.dy), torch.zeros_like(d.s)
    cfg = A.make_conv_cfg(B, L, C, W, act=A.ACT_SILU if d.act else A.ACT_NONE, dtype=CODE[dtype])
    A.atlas_conv_forward(d.x, d.w, d.b, cfg, y, d.s, new)
    for b in range(B):
        d.check(y[b], new[b], (b,), d.sh[b], dtype, f"sequence {b}")
    # in place, and without a state
    same = d.s.clone()
    A.atlas_conv_forward(d.x, d.w, d.b, cfg, y, same, same)
    assert torch.equal(same, new)
    A.atlas_conv_forward(d.x, d.w, d.b, cfg, y, None, None)
    for b in range(B):
        d.check(y[b], None, (b,), 0 * d.sh[b], dtype, f"sequence {b} from zeros")


def test_conv_infinite_input_stays_in_its_window():
    """An infinity reaches W tokens and no more."""
    x = torch.zeros(1, 40, 8, device="cuda")
    x[0, 10, 3] = float("inf")
    w, y = torch.full((8, 3), 0.5, device="cuda"), torch.empty(1, 40, 8, device="cuda")
    A.atlas_conv_forward(x, w, None, A.make_conv_cfg(1, 40, 8, 3, dtype=A.F32), y)
    assert torch.isinf(y).nonzero()[:, 1:].tolist() == [[10, 3], [11, 3], [12, 3]] and not torch.isnan(y).any()


@pytest.mark.parametrize("hd,W", [(16, 4), (12, 4), (8, 3), (5, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_conv_head_major(hd, W, dtype):
    """y in [B, H, L, head_dim], its gradient read from there; packed: [H, rows, head_dim]."""
    B, L, C = 2, 70, hd * 6
    r = rng(6, hd, W)
    d = Conv(r, B, L, C, W, dtype)
    flat, heads = torch.zeros_like(d.x), torch.zeros(B, 6, L, hd, dtype=DT[dtype], device="cuda")
    a, b = A.make_conv_cfg(B, L, C, W, dtype=CODE[dtype]), A.make_conv_cfg(B, L, C, W, dtype=CODE[dtype], head_dim=hd)
    A.atlas_conv_forward(d.x, d.w, d.b, a, flat, d.s)
    A.atlas_conv_forward(d.x, d.w, d.b, b, heads, d.s)
    assert torch.equal(heads, flat.view(B, L, 6, hd).transpose(1, 2))
    out = []
    for cfg, dy in ((a, d.dy), (b, d.dy.view(B, L, 6, hd).transpose(1, 2).contiguous())):
        space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
        o = [torch.zeros_like(d.x), torch.zeros(C, W, device="cuda"), torch.zeros(C, device="cuda"), d.ds.clone()]
        A.atlas_conv_backward(d.x, d.w, d.b, cfg, d.s, dy, o[3], *o[:3])
        out.append(o)
        torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype,C,W", [("bf16", 72, 4), ("fp32", 5, 3), ("fp16", 64, 8)])
def test_conv_packed(lens, dtype, C, W):
    """Slots in another order than the sequences, some from zeros, one padding; rows in front and
    behind untouched; then the backward pass."""
    B = len(lens)
    r = rng(7, *lens, C)
    start, T, at = packed(lens, front=2)
    d = Conv(r, B, 0, C, W, dtype, n=B + 2, packed_rows=T)
    slots = np.roll(np.arange(B), 1) + 1
    pad = B - 1 if B > 2 else None
    if pad is not None:
        slots[pad] = -1
    carry = np.arange(B) % 3 != 1
    st = status()
    cfg = A.make_conv_cfg(B, T, C, W, dtype=CODE[dtype], seq_start=start, slot=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          n_slots=B + 2, carry=torch.tensor(carry, dtype=torch.uint8, device="cuda"), status_dev=st)
    y, new = torch.full_like(d.x, 77.0), d.s.clone()
    A.atlas_conv_forward(d.x, d.w, d.b, cfg, y, new, new)
    used = np.zeros(T, bool)
    left = np.ones(B + 2, bool)
    for b, n in enumerate(lens):
        if slots[b] < 0:
            continue
        rows = slice(at[b], at[b] + n)
        used[rows] = True
        left[slots[b]] = False
        d.check(y[rows], new[slots[b]], rows, d.sh[slots[b]] * carry[b], dtype, f"sequence {b}")
    assert (host(y)[~used] == 77).all() and (host(new)[left] == d.sh[left]).all() and int(st) == 0
    # backward: states by sequence
    cfg = A.make_conv_cfg(B, T, C, W, dtype=CODE[dtype], seq_start=start, carry=torch.tensor(carry, dtype=torch.uint8, device="cuda"))
    space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
    dx, dw, db, ds = torch.full_like(d.x, 77.0), torch.zeros(C, W, device="cuda"), torch.zeros(C, device="cuda"), d.ds.clone()
    A.atlas_conv_backward(d.x, d.w, d.b, cfg, d.s[:B].contiguous(), d.dy, ds, dx, dw, db)
    want, mag = [dict(dw=0, dbias=0) for _ in range(2)]
    for b, n in enumerate(lens):
        rows = slice(at[b], at[b] + n)
        for o, m in ((want, False), (mag, True)):
            g = R.conv_back(d.xh[rows], d.wh, d.bh, True, d.sh[b] * carry[b], d.dyh[rows], d.dsh[b], mag=m)
            o["dw"], o["dbias"] = o["dw"] + g["dw"], o["dbias"] + g["dbias"]
            o[b] = g
        close(dx[rows], want[b]["dx"], mag[b]["dx"], dtype, 0, f"dx {b}")
        close(ds[b], want[b]["dstate"] * carry[b], mag[b]["dstate"], "fp32", 0, f"dstate {b}")
    close(dw, want["dw"], mag["dw"], "fp32", T, "dw")
    close(db, want["dbias"], mag["dbias"], "fp32", T, "dbias")
    assert (host(dx)[:2] == 77).all() and (host(dx)[-3:] == 77).all()


def test_many_packed_sequences():
    """Some 1500 sequences of 0 to 5 tokens: every one finds its rows, its slot and its state."""
    r = rng(25)
    B, C, N, W = 1531, 24, 16, 4
    lens = [int(n) for n in r.integers(0, 6, B)]
    start, T, at = packed(lens)
    slots = r.permutation(B + 7)[:B]
    slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
    st = status()
    c = Conv(r, B, 0, C, W, "fp32", n=B + 7, packed_rows=T)
    y, new = torch.full_like(c.x, 77.0), c.s.clone()
    A.atlas_conv_forward(c.x, c.w, c.b, A.make_conv_cfg(B, T, C, W, dtype=A.F32, seq_start=start, slot=slot, n_slots=B + 7, status_dev=st), y, new, new)
    d = Scan(r, B, 0, C, N, 1, "fp32", n=B + 7, packed_rows=T)
    h = d.h.clone()
    z = run_scan(d, A.make_scan_cfg(B, T, C, N, dtype=A.F32, seq_start=start, slot=slot, n_slots=B + 7, status_dev=st), h, h)
    assert int(st) == 0 and (y[-3:] == 77).all() and (z[-3:] == 77).all()
    y, new, z, h = host(y), host(new), host(z), host(h)
    for b, n in enumerate(lens):
        rows, s = slice(at[b], at[b] + n), slots[b]
        c.check(y[rows], None, rows, c.sh[s], "fp32", f"sequence {b}")
        assert (new[s] == R.conv(c.xh[rows], c.wh, c.bh, True, c.sh[s])[1]).all()
        d.check(z[rows], h[s], rows, d.h_h[s], f"sequence {b}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,C,W,act", [(2, 5, 8, 4, True), (1, 1, 3, 4, True), (2, 2, 40, 4, False), (1, 65, 264, 1, True), (3, 300, 33, 3, True),
                                         (2, 9, 16, 8, True), (1, 3, 16, 8, True), (2, 200, 520, 5, True), (2, 0, 8, 4, True), (0, 5, 8, 4, True)])
def test_conv_backward(B, L, C, W, act, dtype):
    r = rng(8, B, L, C, W)
    d = Conv(r, B, L, C, W, dtype, act=act)
    cfg = A.make_conv_cfg(B, L, C, W, act=A.ACT_SILU if act else A.ACT_NONE, dtype=CODE[dtype])
    space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
    dx, dw, db, ds = torch.zeros_like(d.x), torch.full((C, W), 9.0, device="cuda"), torch.full((C,), 9.0, device="cuda"), d.ds.clone()
    A.atlas_conv_backward(d.x, d.w, d.b, cfg, d.s, d.dy, ds, dx, dw, db)
    want, mag = [dict(dw=np.zeros((C, W)), dbias=np.zeros(C)) for _ in range(2)]
    for b in range(B):
        g, m = (R.conv_back(d.xh[b], d.wh, d.bh, act, d.sh[b], d.dyh[b], d.dsh[b], mag=v) for v in (False, True))
        close(dx[b], g["dx"], m["dx"], dtype, 0, f"dx {b}")
        close(ds[b], g["dstate"], m["dstate"], "fp32", 0, f"dstate {b}")
        for k in ("dw", "dbias"):
            want[k], mag[k] = want[k] + g[k], mag[k] + m[k]
    close(dw, want["dw"], mag["dw"], "fp32", B * L, "dw")
    close(db, want["dbias"], mag["dbias"], "fp32", B * L, "dbias")


# ------------------------------------------------------------------ scan

class Scan:
    def __init__(self, r, B, L, D, N, G, dtype, gate=True, skip=True, bias=True, n=None, packed_rows=None):
        lead = (packed_rows,) if packed_rows else (B, L)
        self.G, self.dtype, self.lead = G, dtype, lead
        for k, shape, s in (("x", (*lead, D), 1), ("dt", (*lead, D), 0.5), ("Bm", (*lead, G, N), 1), ("Cm", (*lead, G, N), 1), ("z", (*lead, D), 1), ("dy", (*lead, D), 1)):
            t, h = draw(r, shape, dtype, s)
            setattr(self, k, t)
            setattr(self, k + "_h", h)
        self.A, self.A_h = (lambda t: (t, host(t)))(dev(-r.uniform(0.3, 1, (D, N)) * np.arange(1, N + 1)))
        self.Dk, self.Dk_h = draw(r, D, "fp32")
        self.bias, self.bias_h = (lambda t: (t, host(t)))(dev(r.uniform(-5, 0, D)))
        self.h, self.h_h = draw(r, (n or B, D, N), "fp32")
        self.dh, self.dh_h = draw(r, (B, D, N), "fp32")
        if not gate:
            self.z = self.z_h = None
        if not skip:
            self.Dk = self.Dk_h = None
        if not bias:
            self.bias = self.bias_h = None
        self.softplus = True

    def inputs(self):
        return self.x, self.dt, self.A, self.Bm, self.Cm, self.Dk, self.z, self.bias

    def ref(self, rows, h0, grad=None, mag=False):
        pick = lambda k: None if getattr(self, k) is None else getattr(self, k + "_h")[rows]  # noqa: E731
        extra = () if grad is None else (self.dy_h[rows], grad)
        return R.scan(pick("x"), pick("dt"), self.A_h, pick("Bm"), pick("Cm"), self.Dk_h, pick("z"), self.bias_h, self.softplus, h0, self.G, *extra, mag=mag)

    def check(self, y, h, rows, h0, what):
        o, S = self.ref(rows, h0), self.ref(rows, h0, mag=True)
        n = o["y"].shape[0] + self.A_h.shape[1]
        close(y, o["y"], S["y"], self.dtype, n, what + " y")
        if h is not None:
            close(h, o["h"], S["h"], "fp32", n, what + " h")

    def grads(self):
        like = dict(dx=self.x, ddt=self.dt, dB=self.Bm, dC=self.Cm, dz=self.z, dA=self.A, dD=self.Dk, ddt_bias=self.bias)
        return {k: None if v is None else torch.full_like(v, 77.0) for k, v in like.items()}

    def backward(self, cfg, h_in, dh):
        space(cfg, A.atlas_scan_backward_workspace_bytes(cfg))
        o = self.grads()
        A.atlas_scan_backward(*self.inputs(), cfg, h_in, self.dy, dh, o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], o["dD"], o["dz"], o["ddt_bias"])
        torch.cuda.synchronize()
        return o


def run_scan(d, cfg, h_in, h_out):
    space(cfg, A.atlas_scan_workspace_bytes(cfg))
    y = torch.full_like(d.x, 77.0)
    A.atlas_scan_forward(*d.inputs(), cfg, y, h_in, h_out)
    torch.cuda.synchronize()
    return y


SCANS = [(2, 5, 8, 4, 1), (1, 1, 3, 1, 1), (5, 1, 64, 16, 1), (3, 1, 40, 13, 2), (2, 31, 40, 8, 1), (1, 33, 33, 13, 1), (2, 64, 64, 16, 2), (1, 70, 96, 16, 3),
         (2, 100, 12, 20, 2), (1, 50, 16, 40, 1), (1, 40, 8, 128, 1), (2, 0, 8, 16, 1), (1, 1000, 72, 16, 1), (2, 517, 34, 5, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,D,N,G", SCANS)
def test_scan(B, L, D, N, G, dtype):
    r = rng(9, B, L, D, N)
    d = Scan(r, B, L, D, N, G, dtype, gate=N != 13, skip=N != 8, bias=N != 20)
    cfg = A.make_scan_cfg(B, L, D, N, G, dtype=CODE[dtype])
    h = torch.zeros_like(d.h)
    y = run_scan(d, cfg, d.h, h)
    for b in range(B):
        d.check(y[b], h[b], (b,), d.h_h[b], f"sequence {b}")
    same = d.h.clone()
    assert torch.equal(run_scan(d, cfg, same, same), y) and torch.equal(same, h)
    y = run_scan(d, cfg, None, None)
    for b in range(B):
        d.check(y[b], None, (b,), 0 * d.h_h[b], f"sequence {b} from zeros")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,L,D,N,G", [(1, 600, 64, 32, 1), (2, 700, 20, 40, 1), (1, 530, 6, 128, 2), (1, 900, 70, 30, 1), (1, 1030, 128, 8, 2)])
def test_scan_segments_of_every_width(B, L, D, N, G, dtype):
    """Several segments a sequence, forward and backward, for each number of lanes a channel."""
    r = rng(26, B, L, D, N)
    d = Scan(r, B, L, D, N, G, dtype)
    cfg = A.make_scan_cfg(B, L, D, N, G, dtype=CODE[dtype])
    assert A.atlas_scan_workspace_bytes(cfg) > 0  # segments
    h = d.h.clone()
    y = run_scan(d, cfg, h, h)
    for b in range(B):
        d.check(y[b], h[b], (b,), d.h_h[b], f"sequence {b}")
    dh = d.dh.clone()
    o = d.backward(A.make_scan_cfg(B, L, D, N, G, dtype=CODE[dtype]), d.h, dh)
    check_grads(d, o, dh, [((b,), d.h_h[b], True) for b in range(B)])


def test_scan_without_softplus_and_large_steps():
    """dt as given; and raw steps whose softplus is the identity or vanishes."""
    r = rng(10)
    d = Scan(r, 2, 60, 24, 16, 1, "fp32", bias=False)
    d.dt = d.dt.abs() * 0.3
    d.dt_h, d.softplus = host(d.dt), False
    h = torch.zeros_like(d.h)
    y = run_scan(d, A.make_scan_cfg(2, 60, 24, 16, dtype=A.F32, softplus=False), d.h, h)
    for b in range(2):
        d.check(y[b], h[b], (b,), d.h_h[b], f"sequence {b}")
    d = Scan(r, 1, 60, 24, 16, 1, "fp32", bias=False)
    d.dt = d.dt * 40
    d.dt_h = host(d.dt)
    y = run_scan(d, A.make_scan_cfg(1, 60, 24, 16, dtype=A.F32), d.h, h[:1])
    d.check(y[0], h[0], (0,), d.h_h[0], "large steps")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_strides(dtype):
    """x, z and dt as slices of wider rows, B and C as slices of another, batch inside token."""
    r = rng(11)
    B, L, D, N = 2, 300, 40, 16
    d = Scan(r, B, L, D, N, 1, dtype)
    wide = torch.zeros(L, B, 3 * D + 8, dtype=DT[dtype], device="cuda")
    small = torch.zeros(B, L, 2 * N + 3, dtype=DT[dtype], device="cuda")
    for i, k in enumerate(("x", "z", "dt")):
        wide[:, :, i * D:(i + 1) * D] = getattr(d, k).transpose(0, 1)
    small[:, :, :N], small[:, :, N + 3:] = d.Bm[:, :, 0], d.Cm[:, :, 0]
    t, s = (wide.stride(1), wide.stride(0)), (small.stride(0), small.stride(1))
    cfg = A.make_scan_cfg(B, L, D, N, dtype=CODE[dtype], x_strides=t, z_strides=t, dt_strides=t, y_strides=t, B_strides=s, C_strides=s)
    space(cfg, A.atlas_scan_workspace_bytes(cfg))
    out = torch.full_like(wide, 77.0)
    y, h = out[:, :, :D], torch.zeros_like(d.h)
    A.atlas_scan_forward(wide[:, :, :D], wide[:, :, 2 * D:3 * D], d.A, small[:, :, :N], small[:, :, N + 3:], d.Dk, wide[:, :, D:2 * D], d.bias, cfg, y, d.h, h)
    for b in range(B):
        d.check(y[:, b], h[b], (b,), d.h_h[b], f"sequence {b}")
    assert (out[:, :, D:] == 77).all()
    # gradients land in slices of the same shapes
    space(cfg, A.atlas_scan_backward_workspace_bytes(cfg))
    g, gs = torch.full_like(wide, 77.0), torch.full_like(small, 77.0)
    out[:, :, :D] = d.dy.transpose(0, 1)
    dA, dD, db, dh = torch.zeros_like(d.A), torch.zeros_like(d.Dk), torch.zeros_like(d.bias), d.dh.clone()
    A.atlas_scan_backward(wide[:, :, :D], wide[:, :, 2 * D:3 * D], d.A, small[:, :, :N], small[:, :, N + 3:], d.Dk, wide[:, :, D:2 * D], d.bias, cfg, d.h,
                          y, dh, g[:, :, :D], g[:, :, 2 * D:3 * D], dA, gs[:, :, :N], gs[:, :, N + 3:], dD, g[:, :, D:2 * D], db)
    plain = d.backward(A.make_scan_cfg(B, L, D, N, dtype=CODE[dtype]), d.h, d.dh.clone())
    for i, k in enumerate(("dx", "dz", "ddt")):
        assert torch.equal(g[:, :, i * D:(i + 1) * D].transpose(0, 1), plain[k]), k
    assert torch.equal(gs[:, :, :N], plain["dB"][:, :, 0]) and torch.equal(gs[:, :, N + 3:], plain["dC"][:, :, 0])
    assert torch.equal(dA, plain["dA"]) and (g[:, :, 3 * D:] == 77).all() and (gs[:, :, N:N + 3] == 77).all()


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype,D,N", [("bf16", 72, 16), ("fp32", 5, 7)])
def test_scan_packed(lens, dtype, D, N):
    B = len(lens)
    r = rng(12, *lens, D)
    start, T, at = packed(lens, front=2)
    d = Scan(r, B, 0, D, N, 1, dtype, n=B + 2, packed_rows=T)
    slots = np.roll(np.arange(B), 1) + 1
    if B > 2:
        slots[B - 1] = -1
    carry = np.arange(B) % 3 != 1
    st = status()
    cfg = A.make_scan_cfg(B, T, D, N, dtype=CODE[dtype], seq_start=start, slot=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                          n_slots=B + 2, carry=torch.tensor(carry, dtype=torch.uint8, device="cuda"), status_dev=st)
    h = d.h.clone()
    y = run_scan(d, cfg, h, h)
    used, left = np.zeros(T, bool), np.ones(B + 2, bool)
    for b, n in enumerate(lens):
        if slots[b] < 0:
            continue
        rows = slice(at[b], at[b] + n)
        used[rows], left[slots[b]] = True, False
        d.check(y[rows], h[slots[b]], rows, d.h_h[slots[b]] * carry[b], f"sequence {b}")
    assert (host(y)[~used] == 77).all() and (host(h)[left] == d.h_h[left]).all() and int(st) == 0
    cfg = A.make_scan_cfg(B, T, D, N, dtype=CODE[dtype], seq_start=start, carry=torch.tensor(carry, dtype=torch.uint8, device="cuda"))
    dh = d.dh.clone()
    o = d.backward(cfg, d.h[:B].contiguous(), dh)
    check_grads(d, o, dh, [(slice(at[b], at[b] + n), d.h_h[b] * carry[b], carry[b]) for b, n in enumerate(lens)])
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        assert (host(o[k])[:2] == 77).all() and (host(o[k])[-3:] == 77).all(), k


def check_grads(d, o, dh, seqs):
    total = {k: [0.0, 0.0] for k in ("dA", "dD", "ddt_bias")}
    T = 0
    for b, (rows, h0, carry) in enumerate(seqs):
        g, S = d.ref(rows, h0, d.dh_h[b]), d.ref(rows, h0, d.dh_h[b], mag=True)
        n = g["y"].shape[0] + d.A_h.shape[1]
        T += n
        for k in ("dx", "ddt", "dz", "dB", "dC"):
            if o[k] is not None:
                close(o[k][rows], g[k], S[k], d.dtype, n + (d.x.shape[-1] if k in ("dB", "dC") else 0), f"{k} of sequence {b}")
        close(dh[b], g["dh"] * carry, S["dh"], "fp32", n, f"dh of sequence {b}")
        for k in total:
            total[k][0], total[k][1] = total[k][0] + g[k], total[k][1] + S[k]
    for k in total:
        if o[k] is not None:
            close(o[k], total[k][0] + 0 * host(o[k]), total[k][1], "fp32", T, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,L,D,N,G", SCANS)
def test_scan_backward(B, L, D, N, G, dtype):
    r = rng(13, B, L, D, N)
    d = Scan(r, B, L, D, N, G, dtype, gate=N != 13, skip=N != 8, bias=N != 20)
    dh = d.dh.clone()
    o = d.backward(A.make_scan_cfg(B, L, D, N, G, dtype=CODE[dtype]), d.h, dh)
    check_grads(d, o, dh, [((b,), d.h_h[b], True) for b in range(B)])
    o = d.backward(A.make_scan_cfg(B, L, D, N, G, dtype=CODE[dtype]), None, None)
    d.dh_h = 0 * d.dh_h
    check_grads(d, o, torch.zeros_like(d.dh), [((b,), 0 * d.h_h[b], False) for b in range(B)])


def test_no_sequences():
    """B = 0, in rows and packed: no gradient, sums of nothing are zero, nothing else is touched."""
    for start in (None, torch.zeros(1, dtype=torch.int32, device="cuda")):
        d = Scan(rng(23), 1, 0, 16, 16, 1, "fp32", packed_rows=8)
        cfg = A.make_scan_cfg(0, 8, 16, 16, dtype=A.F32, seq_start=start)
        o = d.backward(cfg, None, None)
        assert not o["dA"].any() and not o["dD"].any() and not o["ddt_bias"].any()
        assert all((o[k] == 77).all() for k in ("dx", "ddt", "dB", "dC", "dz"))
        assert (run_scan(d, cfg, None, None) == 77).all()


def test_scan_against_differences():
    """The forward's own differences, in 32 bits: L(x + e d) - L(x - e d) over 2e is g.d to e^2 and
    to the rounding of the losses, |L| 2^-20 / e."""
    r = rng(14)
    d = Scan(r, 2, 40, 16, 16, 1, "fp32")
    cfg = A.make_scan_cfg(2, 40, 16, 16, dtype=A.F32)
    dh = d.dh.clone()
    o = d.backward(cfg, d.h, dh)

    def loss():
        h = torch.zeros_like(d.h)
        y = run_scan(d, cfg, d.h, h)
        return (float((y.double() * d.dy.double()).sum() + (h.double() * d.dh.double()).sum()),
                float((y.double() * d.dy.double()).abs().sum() + (h.double() * d.dh.double()).abs().sum()))
    e = 2.0 ** -8
    for k, g in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("Dk", "dD"), ("z", "dz"), ("bias", "ddt_bias")):
        v = getattr(d, k)
        way = dev(r.standard_normal(v.shape)) / v.numel() ** 0.5
        vals = []
        for s in (e, -e):
            setattr(d, k, v + s * way)
            vals.append(loss())
        setattr(d, k, v)
        want = float((o[g].double() * way.double()).sum())
        scale = float((o[g].double().abs() * way.double().abs()).sum())
        got = (vals[0][0] - vals[1][0]) / (2 * e)
        assert abs(got - want) <= 0.02 * scale + vals[0][1] * 2.0 ** -20 / e, (k, got, want)


# ------------------------------------------------- slots, tokens, streams, graphs

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [1, 6])
def test_bad_slots_are_left_out(dtype, L):
    """An index past the pool, and the second use of one: nothing of those sequences is touched,
    the status says so, the others are computed."""
    B, D, N, W = 6, 40, 16, 4
    r = rng(15, L)
    slots = torch.tensor([3, 9, 0, 3, -1, 1], dtype=torch.int32, device="cuda")
    good = [0, 2, 5]
    st = status()
    d = Scan(r, B, L, D, N, 1, dtype, n=4)
    cfg = A.make_scan_cfg(B, L, D, N, dtype=CODE[dtype], slot=slots, n_slots=4, status_dev=st)
    h = d.h.clone()
    y = run_scan(d, cfg, h, h)
    assert int(st) == A.ERR_INVALID
    for b in range(B):
        if b in good:
            d.check(y[b], h[slots[b]], (b,), d.h_h[int(slots[b])], f"sequence {b}")
        else:
            assert (y[b] == 77).all()
    assert torch.equal(h[2], d.h[2])
    st.zero_()
    c = Conv(r, B, L, D, W, dtype, n=4)
    cfg = A.make_conv_cfg(B, L, D, W, dtype=CODE[dtype], slot=slots, n_slots=4, status_dev=st)
    y, new = torch.full_like(c.x, 77.0), c.s.clone()
    A.atlas_conv_forward(c.x, c.w, c.b, cfg, y, new, new)
    assert int(st) == A.ERR_INVALID
    for b in range(B):
        if b in good:
            c.check(y[b], new[slots[b]], (b,), c.sh[int(slots[b])], dtype, f"sequence {b}")
        else:
            assert (y[b] == 77).all()
    assert torch.equal(new[2], c.s[2])


@pytest.mark.parametrize("start", [[0, 5, 3, 9], [0, 4, 8, 99], [-3, 2, 4, 8]])
def test_bad_starts_are_left_out(start):
    """Packed starts that fall back, pass the rows or are negative: reported, the valid sequences computed."""
    r, T, st = rng(16), 12, status()
    t = torch.tensor(start, dtype=torch.int32, device="cuda")
    d = Scan(r, 3, 0, 16, 16, 1, "fp32", packed_rows=T)
    run_scan(d, A.make_scan_cfg(3, T, 16, 16, dtype=A.F32, seq_start=t, status_dev=st), d.h, d.h.clone())
    assert int(st) == A.ERR_INVALID
    st.zero_()
    c = Conv(r, 3, 0, 16, 4, "fp32", packed_rows=T)
    y = torch.full_like(c.x, 77.0)
    A.atlas_conv_forward(c.x, c.w, c.b, A.make_conv_cfg(3, T, 16, 4, dtype=A.F32, seq_start=t, status_dev=st), y, c.s, c.s.clone())
    assert int(st) == A.ERR_INVALID


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_tokens_continue_a_prompt(dtype):
    """A prompt and then single tokens give what the whole sequence gives: the convolution bit
    for bit, the scan to its tolerance (segments add in another order)."""
    r = rng(17)
    B, L, n, D, N, W = 2, 300, 4, 48, 16, 4
    d, c = Scan(r, B, L + n, D, N, 1, dtype), Conv(r, B, L + n, D, W, dtype)
    h, s = d.h.clone(), c.s.clone()
    ys, yc = torch.full_like(d.x, 77.0), torch.full_like(c.x, 77.0)
    for lo, hi in [(0, L)] + [(L + i, L + i + 1) for i in range(n)]:
        t = (d.x.stride(0), d.x.stride(1))
        bc = (d.Bm.stride(0), d.Bm.stride(1))
        cfg = A.make_scan_cfg(B, hi - lo, D, N, dtype=CODE[dtype], x_strides=t, dt_strides=t, z_strides=t, y_strides=t, B_strides=bc, C_strides=bc)
        space(cfg, A.atlas_scan_workspace_bytes(cfg))
        v = lambda k: k[:, lo:hi]  # noqa: E731
        A.atlas_scan_forward(v(d.x), v(d.dt), d.A, v(d.Bm), v(d.Cm), d.Dk, v(d.z), d.bias, cfg, v(ys), h, h)
        ccfg = A.make_conv_cfg(B, hi - lo, D, W, dtype=CODE[dtype], x_strides=t, y_strides=t)
        A.atlas_conv_forward(v(c.x), c.w, c.b, ccfg, v(yc), s, s)
        torch.cuda.synchronize()
    for b in range(B):
        d.check(ys[b], h[b], (b,), d.h_h[b], f"sequence {b}")
    whole, new = torch.empty_like(c.x), torch.empty_like(c.s)
    A.atlas_conv_forward(c.x, c.w, c.b, A.make_conv_cfg(B, L + n, D, W, dtype=CODE[dtype]), whole, c.s, new)
    assert torch.equal(whole, yc) and torch.equal(new, s)


def test_same_bits_on_streams_and_in_graphs():
    """Forward and backward of all three on a side stream, captured into a graph and replayed on
    new inputs: the bits of the plain calls."""
    r = rng(18)
    d, c = Scan(r, 2, 400, 64, 16, 1, "bf16"), Conv(r, 2, 400, 64, 4, "bf16")
    hx, _ = draw(r, (50, 256), "bf16")
    w, _ = draw(r, 256, "bf16")
    scfg, ccfg, ncfg = A.make_scan_cfg(2, 400, 64, 16), A.make_conv_cfg(2, 400, 64, 4), A.make_norm_cfg(50, 256)
    fcfg = A.make_scan_cfg(2, 400, 64, 16)
    space(scfg, A.atlas_scan_backward_workspace_bytes(scfg))
    space(ccfg, A.atlas_conv_backward_workspace_bytes(ccfg))
    space(ncfg, A.atlas_norm_backward_workspace_bytes(ncfg))
    space(fcfg, A.atlas_scan_workspace_bytes(fcfg))
    o = d.grads()
    o.update(y=torch.zeros_like(d.x), h=torch.zeros_like(d.h), dh=d.dh.clone(), cy=torch.zeros_like(c.x), cs=torch.zeros_like(c.s), cdx=torch.zeros_like(c.x),
             cdw=torch.zeros(64, 4, device="cuda"), cdb=torch.zeros(64, device="cuda"), cds=c.ds.clone(), ny=torch.zeros_like(hx), ndx=torch.zeros_like(hx), ndw=torch.zeros(256, device="cuda"))

    def everything():
        o["dh"].copy_(d.dh)
        o["cds"].copy_(c.ds)
        A.atlas_scan_forward(*d.inputs(), fcfg, o["y"], d.h, o["h"])
        A.atlas_scan_backward(*d.inputs(), scfg, d.h, d.dy, o["dh"], o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], o["dD"], o["dz"], o["ddt_bias"])
        A.atlas_conv_forward(c.x, c.w, c.b, ccfg, o["cy"], c.s, o["cs"])
        A.atlas_conv_backward(c.x, c.w, c.b, ccfg, c.s, c.dy, o["cds"], o["cdx"], o["cdw"], o["cdb"])
        A.atlas_norm_forward(hx, None, w, ncfg, o["ny"])
        A.atlas_norm_backward(hx, w, o["ny"], None, ncfg, o["ndx"], o["ndw"])
    everything()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    torch.cuda.synchronize()  # the copies are ordered on the default stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        everything()
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], o[k]) for k in o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything()
    for t in (d.x, c.x, hx):
        t.mul_(0.5)
    everything()
    torch.cuda.synchronize()
    second = {k: v.clone() for k, v in o.items()}
    for v in o.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(second[k], o[k]) for k in o) and not torch.equal(first["y"], second["y"])


def test_tensors_that_do_not_fit_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    y, cfg = torch.zeros_like(x), A.make_norm_cfg(4, 64)
    for bad in (x.float(), x.cpu(), x[:3], x.flatten()[:255]):
        with pytest.raises(A.AtlasError):
            A.atlas_norm_forward(bad, None, None, cfg, y)
    A.atlas_norm_forward(x, None, None, cfg, y)
    # a strided view whose storage reaches far enough passes, one row more does not
    wide = torch.zeros(4, 80, dtype=torch.bfloat16, device="cuda")
    A.atlas_norm_forward(wide[:, :64], None, None, A.make_norm_cfg(4, 64, x_stride=80), y)
    with pytest.raises(A.AtlasError):
        A.atlas_norm_forward(wide[:, :64], None, None, A.make_norm_cfg(5, 64, x_stride=80), torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda"))
    for name, t in (("seq_start", torch.zeros(2, dtype=torch.int64, device="cuda")), ("slot", torch.zeros(1, dtype=torch.int32, device="cuda")),
                    ("carry", torch.zeros(2, dtype=torch.bool, device="cuda")), ("seq_start", torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(A.AtlasError):
            A.make_conv_cfg(2, 4, 8, 4, **{name: t})


def test_conv_rows_past_32_bits():
    """More than 2^32 elements: the last rows as they are in a short sequence."""
    C, W = 2048, 4
    L = (1 << 32) // C + 11
    x = torch.zeros(1, L, C, dtype=torch.bfloat16, device="cuda")
    x[0, -20:] = dev(rng(19).standard_normal((20, C)), "bf16")
    w, _ = draw(rng(20), (C, W), "bf16")
    y, s = torch.empty_like(x), torch.empty(1, W - 1, C, dtype=torch.bfloat16, device="cuda")
    A.atlas_conv_forward(x, w, None, A.make_conv_cfg(1, L, C, W), y, None, s)
    one, s1 = torch.empty(1, 20, C, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s)
    A.atlas_conv_forward(x[:, -20:], w, None, A.make_conv_cfg(1, 20, C, W), one, None, s1)
    assert torch.equal(y[:, -20:], one) and torch.equal(s, s1) and not y[0, :-20:997].any()


def test_scan_rows_past_32_bits():
    """More than 2^32 elements in one sequence of many segments: zeros up to the last 20 tokens,
    which are as they are alone."""
    D, N = 2048, 4
    L = (1 << 32) // D + 21
    r = rng(22)
    d = Scan(r, 1, 20, D, N, 1, "bf16", gate=False)
    big = [torch.zeros(1, L, *t.shape[2:], dtype=t.dtype, device="cuda") for t in (d.x, d.dt, d.Bm, d.Cm)]
    for t, s in zip(big, (d.x, d.dt, d.Bm, d.Cm)):
        t[:, -20:] = s
    y, h, one, h1 = torch.empty_like(big[0]), torch.empty(1, D, N, device="cuda"), torch.empty_like(d.x), torch.empty(1, D, N, device="cuda")
    for x, dt, Bm, Cm, n, out, state in ((*big, L, y, h), (d.x, d.dt, d.Bm, d.Cm, 20, one, h1)):
        cfg = A.make_scan_cfg(1, n, D, N)
        space(cfg, A.atlas_scan_workspace_bytes(cfg))
        A.atlas_scan_forward(x, dt, d.A, Bm, Cm, d.Dk, None, d.bias, cfg, out, None, state)
        torch.cuda.synchronize()
    assert torch.equal(y[:, -20:], one) and torch.equal(h, h1) and not y[0, :-20:997].any()


def test_arguments_that_have_to_be_contiguous():
    """A transposed weight, state or default-stride input has the right number of elements in the
    wrong order."""
    x, w = torch.zeros(2, 16, 8, device="cuda"), torch.zeros(4, 8, device="cuda").t()
    cfg, y, st = A.make_conv_cfg(2, 16, 8, 4, dtype=A.F32), torch.zeros(2, 16, 8, device="cuda"), torch.zeros(2, 8, 3, device="cuda").transpose(1, 2)
    good = w.contiguous()
    for args in ((x, w, None, cfg, y), (x.transpose(0, 1).contiguous().transpose(0, 1), good, None, cfg, y), (x, good, None, cfg, y, st)):
        with pytest.raises(A.AtlasError):
            A.atlas_conv_forward(*args)
    A.atlas_conv_forward(x, good, None, cfg, y, st.contiguous())
    with pytest.raises(A.AtlasError):  # a workspace smaller than it is said to be
        A.make_scan_cfg(1, 4, 8, 4, workspace=torch.zeros(16, device="cuda"), workspace_bytes=65)
    with pytest.raises(A.AtlasError):  # a dimension changed after the description was used
        cfg.L = 17
        A.atlas_conv_forward(x, good, None, cfg, y)


# ------------------------------------------------------- a layer around the memory

def test_layer_around_the_memory_update():
    """Residual and norm, projections, the short convolution of q, k, v written head by head, the
    norm of each key and query, the memory update; beside it the scan on the same normed rows.
    Each step is compared with its definition on the values the step before really gave."""
    import oracle
    import workloads as Wk
    from parity_util import oracle_cfg, rel_err, tol
    from test_memorization_recurrent_gb300.harness import Runner
    r = rng(21)
    B, H, N, d = 1, 2, 130, 128
    C = H * d
    x, xh = draw(r, (B * N, C), "bf16")
    res, rh = draw(r, (B * N, C), "fp32")
    wn, wh = draw(r, C, "bf16")
    y = torch.empty_like(x)
    A.atlas_norm_forward(x, res, wn, A.make_norm_cfg(B * N, C, r_dtype=A.F32), y, res)
    h, want = R.norm(xh, rh, wh, 1e-6)
    close(y, want, np.abs(want), "bf16", 0, "normed rows")
    close(res, h, np.abs(xh) + np.abs(rh), "fp32", 0, "residual")
    proj = [draw(r, (C, C), "bf16", C ** -0.5)[0] for _ in range(3)]
    taps = [draw(r, (C, 4), "bf16", 0.5) for _ in range(3)]
    state = [torch.zeros(B, 3, C, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    unit = torch.full((d,), d ** -0.5, dtype=torch.float32, device="cuda")
    dev_in, ccfg = {}, A.make_conv_cfg(B, N, C, 4, head_dim=d)
    ncfg = A.make_norm_cfg(B * H * N, d, w_dtype=A.F32, eps=0.0)
    for name, p, (t, th), s in zip("QKV", proj, taps, state):
        rows = (y @ p).view(B, N, C)
        out = torch.empty(B, H, N, d, dtype=torch.bfloat16, device="cuda")
        A.atlas_conv_forward(rows, t, None, ccfg, out, s, s)
        ref, _ = R.conv(host(rows)[0], th, None, True, np.zeros((3, C)))
        S, _ = R.conv(host(rows)[0], th, None, True, np.zeros((3, C)), mag=True)
        close(out[0].transpose(0, 1).reshape(N, C), ref, 1.1 * S, "bf16", 0, name)
        if name != "V":
            u = torch.empty_like(out)
            A.atlas_norm_forward(out, None, unit, ncfg, u)
            n = host(u).reshape(-1, d)
            assert np.abs(np.linalg.norm(n, axis=1) - 1).max() < 2.0 ** -8
            out = u
        dev_in[name] = out
    w = Wk.workload(2, B=B, H=H, N=N)
    g = Wk.generate(w)
    inp = {k: host(dev_in[k])[0] for k in "QKV"}
    run = Runner(w, H, N)
    data = {k: dev_in[k][0] for k in "QKV"}
    data.update({k: torch.from_numpy(g[k]).cuda() for k in ("alpha", "eta", "theta", "gamma", "M0")})
    Y, M = run(data)
    torch.cuda.synchronize()
    Yo, Mo, _ = oracle.forward(oracle_cfg(w, N), inp["K"], inp["Q"], inp["V"], g["alpha"], g["eta"], g["theta"], g["gamma"], g["M0"])
    assert rel_err(host(Y), Yo, True) <= tol(w) and rel_err(host(M), Mo, True) <= tol(w)
    # the memory's fp32 output joins the residual stream of the next layer's norm, in 8 bits
    mixed = Y.transpose(0, 1).reshape(B * N, C).contiguous()
    before = host(res)
    q, scale = torch.empty(B * N, C, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(B * N, 2, device="cuda")
    A.atlas_norm_forward(mixed, res, wn, A.make_norm_cfg(B * N, C, dtype=A.F32, r_dtype=A.F32, w_dtype=A.BF16, out_dtype=A.E4M3, group=128), q, res, scale)
    h, want = R.norm(host(mixed), before, wh, 1e-6)
    got = host(q).reshape(B * N, 2, 128) * host(scale)[..., None]
    step = np.abs(want).reshape(B * N, 2, 128)
    assert (np.abs(got - want.reshape(got.shape)) <= 2.0 ** -4 * step * 1.001 + 2.0 ** -10 * host(scale)[..., None] + 1e-5).all()
    # the scan on the same rows
    s = Scan(r, B, N, C, 16, 1, "bf16")
    s.x, s.x_h = y.view(B, N, C), host(y).reshape(B, N, C)
    hs = torch.zeros_like(s.h)
    ys = run_scan(s, A.make_scan_cfg(B, N, C, 16), s.h, hs)
    s.check(ys[0], hs[0], (0,), s.h_h[0], "scan")
