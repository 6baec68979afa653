"""Layer operators where they are easily wrong: 8-bit outputs beside 32-bit ones, norms without
eps, rows past the last, states that are not finite, starts that fall, layouts whose
dimensions lie in any order, batches of many sequences.  References and tolerances as in
test_gpu_layer_ops.py."""
import numpy as np
import pytest

import layer_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_layer_ops import CODE, DT, TYPES, Conv, Scan, _lib, check_grads, close, dev, draw, host, rng, run_scan, space, status  # noqa: E402,F401

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


@pytest.mark.parametrize("dtype,r_dtype", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,d", [(6, 128), (1500, 128), (6, 1000), (1300, 1032), (6, 37), (1300, 1371), (3, 8200), (1, 1)])
def test_rows_of_zeros_without_eps(rows, d, dtype, r_dtype):
    """eps = 0: a row of zeros gives zeros in every output type, and its gradient is what reaches the
    residual stream; it adds nothing to dw."""
    r = rng(32, rows, d)
    x, res, w = draw(r, (rows, d), dtype)[0], draw(r, (rows, d), r_dtype, 2.0)[0], draw(r, d, dtype)[0]
    zero = np.arange(rows) % 3 == 0
    x[torch.from_numpy(zero).cuda()] = 0
    res[torch.from_numpy(zero).cuda()] = 0
    kw = dict(dtype=CODE[dtype], r_dtype=CODE[r_dtype], w_dtype=CODE[dtype], eps=0.0)
    some = np.where(zero[:, None], 1.0, host(x) + host(res))  # (any finite row in the place of zeros)
    want = np.where(zero[:, None], 0.0, R.norm(some, None, host(w), 0.0)[1])
    for out in (dtype, "fp32"):
        y = torch.empty(rows, d, dtype=DT[out], device="cuda")
        A.atlas_norm_forward(x, res, w, A.make_norm_cfg(rows, d, out_dtype=CODE[out], **kw), y)
        close(y, want, np.abs(want), out, 0, out)
    for group in (0, 32):
        g = group if 0 < group < d else d
        q, scale = torch.empty(rows, d, dtype=DT["e4m3"], device="cuda"), torch.empty(rows, -(-d // g), device="cuda")
        A.atlas_norm_forward(x, res, w, A.make_norm_cfg(rows, d, out_dtype=A.E4M3, group=group, **kw), q, None, scale)
        ref = np.maximum(np.stack([np.abs(want[:, i:i + g]).max(1) for i in range(0, d, g)], 1), 1e-30) / 448
        assert (np.abs(host(scale) - ref) <= 2.0 ** -18 * ref).all()
        v = want / np.repeat(ref, g, 1)[:, :d]
        close(q, v, np.abs(v), "e4m3", 0, "q")
    h = dev(host(x) + host(res), r_dtype)
    dy, dh = draw(r, (rows, d), dtype)[0], draw(r, (rows, d), r_dtype)[0]
    hh = np.where(zero[:, None], 1.0, host(h))
    for up in (dh, None):
        cfg = A.make_norm_cfg(rows, d, **kw)
        space(cfg, A.atlas_norm_backward_workspace_bytes(cfg))
        dx, dw = torch.empty_like(h), torch.empty(d, device="cuda")
        A.atlas_norm_backward(h, w, dy, up, cfg, dx, dw)
        uph = np.zeros((rows, d)) if up is None else host(up)
        ref, mag = (R.norm_back(hh, host(w), host(dy), uph, 0.0, mag=m)[0] for m in (False, True))
        close(dx, np.where(zero[:, None], uph, ref), mag, r_dtype, 0, "dx")
        ref, mag = (R.norm_back(hh[~zero], host(w), host(dy)[~zero], None, 0.0, mag=m)[1] if (~zero).any() else np.zeros(d) for m in (False, True))
        close(dw, ref, mag, "fp32", rows / 32, "dw")


@pytest.mark.parametrize("dtype,C", [("bf16", 72), ("fp32", 5)])
def test_conv_gradient_of_states_that_are_not_finite(dtype, C):
    """An empty sequence has no term of dw, whatever its state holds; and the tap of the current token has
    none of any state."""
    r, W = rng(33, C), 4
    start = torch.tensor([0, 20, 20, 29], dtype=torch.int32, device="cuda")
    d = Conv(r, 3, 0, C, W, dtype, act=False, packed_rows=29)
    cfg = A.make_conv_cfg(3, 29, C, W, act=A.ACT_NONE, dtype=CODE[dtype], seq_start=start)
    space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
    out = []
    for bad in (None, 1, 0):
        s = d.s.clone()
        if bad is not None:
            s[bad] = float("nan")
        o = [torch.zeros_like(d.x), torch.zeros(C, W, device="cuda"), torch.zeros(C, device="cuda"), d.ds.clone()]
        A.atlas_conv_backward(d.x, d.w, d.b, cfg, s, d.dy, o[3], *o[:3])
        out.append(o)
        torch.cuda.synchronize()
    plain, empty, first = out
    assert all(torch.equal(p, q) for p, q in zip(plain, empty))
    assert torch.equal(empty[3][1], d.ds[1])
    assert torch.equal(plain[1][:, W - 1], first[1][:, W - 1]) and torch.isnan(first[1][:, :W - 1]).all()


STARTS = [[0, 1000, 200, 1200], [0, 700, 900, 400, 1300], [-3, 600, 1200], [0, 600, 5000], [0, 600, 5000, 900], [5, 3, 1300], [0, 0, 1300, 1299, 1300],
          [4 * i for i in range(200)] + [796, 3] + [5 * i for i in range(120)]]


@pytest.mark.parametrize("start", STARTS)
@pytest.mark.parametrize("dtype,C,N", [("fp32", 5, 7), ("bf16", 72, 16)])
def test_starts_that_fall(start, dtype, C, N):
    """Sequences of several tiles and segments: those in front of the first fall whose rows are there are
    computed, state too; rows and states of the others stay as they are."""
    T, B, W = 1300, len(start) - 1, 4
    fall = next((b for b in range(B) if start[b + 1] < start[b]), B)
    good = [b for b in range(fall) if start[b] >= 0 and start[b + 1] <= T]
    r = rng(36, B, C)
    slots = r.permutation(B + 3)[:B]
    slot, t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (slots, start))
    used, kept = np.zeros(T, bool), np.ones(B + 3, bool)
    for b in good:
        used[start[b]:start[b + 1]], kept[slots[b]] = True, False
    st, d = status(), Scan(r, B, 0, C, N, 1, dtype, n=B + 3, packed_rows=T)
    cfg = A.make_scan_cfg(B, T, C, N, dtype=CODE[dtype], seq_start=t, slot=slot, n_slots=B + 3, status_dev=st)
    assert A.atlas_scan_workspace_bytes(cfg) > 0  # segments
    h = d.h.clone()
    y = run_scan(d, cfg, h, h)
    assert int(st) == A.ERR_INVALID
    for b in good:
        rows = slice(start[b], start[b + 1])
        d.check(y[rows], h[slots[b]], rows, d.h_h[slots[b]], f"sequence {b}")
    assert (host(y)[~used] == 77).all() and (host(h)[kept] == d.h_h[kept]).all()
    st.zero_()
    c = Conv(r, B, 0, C, W, dtype, n=B + 3, packed_rows=T)
    cfg = A.make_conv_cfg(B, T, C, W, dtype=CODE[dtype], seq_start=t, slot=slot, n_slots=B + 3, status_dev=st)
    y, new = torch.full_like(c.x, 77.0), c.s.clone()
    A.atlas_conv_forward(c.x, c.w, c.b, cfg, y, new, new)
    assert int(st) == A.ERR_INVALID
    for b in good:
        rows = slice(start[b], start[b + 1])
        c.check(y[rows], new[slots[b]], rows, c.sh[slots[b]], dtype, f"sequence {b}")
    assert (host(y)[~used] == 77).all() and (host(new)[kept] == c.sh[kept]).all()
    # backward: reported, and nothing outside the rows is written
    st.zero_()
    cfg = A.make_conv_cfg(B, T, C, W, dtype=CODE[dtype], seq_start=t, status_dev=st)
    space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
    dx, ds = torch.full_like(c.x, 77.0), c.ds.clone()
    A.atlas_conv_backward(c.x, c.w, c.b, cfg, c.s[:B].contiguous(), c.dy, ds, dx, torch.zeros(C, W, device="cuda"), torch.zeros(C, device="cuda"))
    assert int(st) == A.ERR_INVALID and (host(dx)[~used] == 77).all()
    assert all((host(ds)[b] == c.dsh[b]).all() for b in range(B) if b not in good)
    st.zero_()
    cfg = A.make_scan_cfg(B, T, C, N, dtype=CODE[dtype], seq_start=t, status_dev=st)
    dh = d.dh.clone()
    o = d.backward(cfg, d.h[:B].contiguous(), dh)
    assert int(st) == A.ERR_INVALID and (host(o["dx"])[~used] == 77).all()
    assert all((host(dh)[b] == d.dh_h[b]).all() for b in range(B) if b not in good)


def device_us(f, n=5):
    """Least time of a call on the device, of n after two."""
    t = []
    for _ in range(n + 2):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        t.append(a.elapsed_time(b) * 1e3)
    return min(t[2:])


@pytest.mark.parametrize("back", [False, True])
def test_conv_time_goes_by_rows(back):
    """65536 rows in 256 sequences, equal ones or one of half the rows, take about as long as in eight
    (a share of work that goes by the number of sequences would make it many times as long)."""
    T, C, W = 65536, 2048, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    x, dy = (torch.randn(T, C, generator=g, device="cuda").bfloat16() for _ in range(2))
    w, b = torch.randn(C, W, generator=g, device="cuda").bfloat16(), torch.randn(C, generator=g, device="cuda").bfloat16()
    y, dw, db = torch.empty_like(x), torch.empty(C, W, device="cuda"), torch.empty(C, device="cuda")
    us = {}
    for name, lens in (("eight", [T // 8] * 8), ("equal", [256] * 256), ("half", [T // 2] + [T // 2 // 255] * 254 + [T // 2 - 254 * (T // 2 // 255)])):
        B = len(lens)
        start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        s = torch.randn(B, W - 1, C, generator=g, device="cuda").bfloat16()
        cfg = A.make_conv_cfg(B, T, C, W, seq_start=start)
        if back:
            space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
            us[name] = device_us(lambda: A.atlas_conv_backward(x, w, b, cfg, s, dy, None, y, dw, db))
        else:
            us[name] = device_us(lambda: A.atlas_conv_forward(x, w, b, cfg, y, s))
    print({k: round(v) for k, v in us.items()})
    assert max(us.values()) <= 1.5 * us["eight"], us


def test_lengths_next_to_2_to_the_31():
    """Rows up to the largest int: the last ones as they are in a short sequence."""
    L, n, W = 2 ** 31 - 1, 50, 3
    r = rng(35)
    x = torch.zeros(L, 1, dtype=torch.bfloat16, device="cuda")
    x[-n:] = dev(r.standard_normal((n, 1)), "bf16")
    w, dy = draw(r, (1, W), "bf16")[0], torch.zeros_like(x)
    dy[-n:] = dev(r.standard_normal((n, 1)), "bf16")
    got = []
    for rows in (L, n):
        y, s = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda"), torch.empty(1, W - 1, 1, dtype=torch.bfloat16, device="cuda")
        A.atlas_conv_forward(x[-rows:], w, None, A.make_conv_cfg(1, rows, 1, W), y, None, s)
        cfg = A.make_conv_cfg(1, rows, 1, W)
        space(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
        dx, dw = torch.empty_like(y), torch.empty(1, W, device="cuda")
        A.atlas_conv_backward(x[-rows:], w, None, cfg, None, dy[-rows:], None, dx, dw, None)
        torch.cuda.synchronize()
        got.append((y[-n:].clone(), s, dx[-n:].clone(), dw))
    assert all(torch.equal(a, b) for a, b in zip(got[0][:3], got[1][:3]))
    xs = host(x[-n:])
    mag = R.conv_back(xs, host(w), None, True, np.zeros((W - 1, 1)), host(dy[-n:]), None, mag=True)
    close(got[0][3], host(got[1][3]), mag["dw"], "fp32", n, "dw")
    del y, dx, dy
    # one channel, one state
    dt, Bm, Cm = (torch.zeros(L, 1, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for t in (dt, Bm, Cm):
        t[-n:] = dev(r.standard_normal((n, 1)), "bf16")
    a, got = torch.full((1, 1), -0.5, device="cuda"), []
    for rows in (L, n):
        cfg = A.make_scan_cfg(1, rows, 1, 1)
        space(cfg, A.atlas_scan_workspace_bytes(cfg))
        y, h = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 1, device="cuda")
        A.atlas_scan_forward(x[-rows:], dt[-rows:], a, Bm[-rows:], Cm[-rows:], None, None, None, cfg, y, None, h)
        torch.cuda.synchronize()
        got.append((y[-n:].clone(), h))
    dth, Bh, Ch = (host(t[-n:]) for t in (dt, Bm, Cm))
    ref, mag = (R.scan(xs, dth, host(a), Bh[:, None], Ch[:, None], None, None, None, True, np.zeros((1, 1)), 1, mag=m) for m in (False, True))
    for y, h in got:
        close(y, ref["y"], mag["y"], "bf16", n + 1, "y")
        close(h[0], ref["h"], mag["h"], "fp32", n + 1, "h")


@pytest.mark.parametrize("order", ["LBHd", "HBLd", "HLBd", "BLHd", "LHBd", "BHLd"])
@pytest.mark.parametrize("B,L,H,hd,dtype", [(3, 37, 4, 8, "bf16"), (2, 20, 3, 5, "fp32"), (2, 1, 4, 8, "bf16"), (1, 9, 4, 8, "fp32")])
def test_conv_heads_in_any_order(order, B, L, H, hd, dtype):
    """y with batch, tokens and heads nested in any order, each with room to spare; dy read from there."""
    r, W, C = rng(34, B, L, H), 4, H * hd
    d = Conv(r, B, L, C, W, dtype)
    size = dict(B=B, L=L, H=H, d=hd)
    wide = torch.full([size[k] + (k == "H") for k in order[:3]] + [hd + 3], 77.0, dtype=DT[dtype], device="cuda")
    y = wide.permute(*(order.index(k) for k in "BLHd"))[:, :, :H, :hd]
    strides = (y.stride(0), y.stride(1), y.stride(2))
    cfg = A.make_conv_cfg(B, L, C, W, dtype=CODE[dtype], head_dim=hd, y_strides=strides)
    A.atlas_conv_forward(d.x, d.w, d.b, cfg, y, d.s)
    flat = torch.empty_like(d.x)
    A.atlas_conv_forward(d.x, d.w, d.b, A.make_conv_cfg(B, L, C, W, dtype=CODE[dtype]), flat, d.s)
    assert torch.equal(y, flat.view(B, L, H, hd)) and int((wide != 77).sum()) <= y.numel()
    y.copy_(d.dy.view(B, L, H, hd))
    out = []
    for c, dy in ((cfg, y), (A.make_conv_cfg(B, L, C, W, dtype=CODE[dtype]), d.dy)):
        space(c, A.atlas_conv_backward_workspace_bytes(c))
        o = [torch.zeros_like(d.x), torch.zeros(C, W, device="cuda"), torch.zeros(C, device="cuda"), d.ds.clone()]
        A.atlas_conv_backward(d.x, d.w, d.b, c, d.s, dy, o[3], *o[:3])
        out.append(o)
        torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][3], out[1][3])
    mag = sum(R.conv_back(d.xh[b], d.wh, d.bh, True, d.sh[b], d.dyh[b], d.dsh[b], mag=True)["dw"] for b in range(B))
    close(out[0][1], host(out[1][1]), mag, "fp32", B * L, "dw")


@pytest.mark.parametrize("L", [1, 20, 700])
def test_scan_decay_next_to_the_largest_number(L):
    """A of -3e38 forgets at once, and leaves the state alone where dt is 0 (raw steps of -200, and places
    behind a sequence's end): its product with log2(e) is not a 32-bit number."""
    r = rng(37, L)
    d = Scan(r, 2, L, 24, 16, 1, "fp32")
    d.A[:, 0], d.A_h[:, 0] = -3e38, float(np.float32(-3e38))
    steps = d.dt.clone(), d.dt_h.copy()
    d.dt[:, L // 2], d.dt_h[:, L // 2] = -200, -200
    d.bias, d.bias_h = None, None
    cfg = A.make_scan_cfg(2, L, 24, 16, dtype=A.F32)
    h = torch.zeros_like(d.h)
    y = run_scan(d, cfg, d.h, h)
    for b in range(2):
        d.check(y[b], h[b], (b,), d.h_h[b], f"sequence {b}")
    (d.dt, d.dt_h), dh = steps, d.dh.clone()  # (at a step of 0 the gradient's A times a state is no number of 32 bits)
    o = d.backward(A.make_scan_cfg(2, L, 24, 16, dtype=A.F32), d.h, dh)
    check_grads(d, o, dh, [((b,), d.h_h[b], True) for b in range(2)])


def test_graphs_replayed_on_other_starts():
    """Forward and backward of packed convolutions and scans of many sequences, captured, and replayed after
    the starts have changed in place: the bits of plain calls on them."""
    r, B, T, C, N, W = rng(38), 100, 1400, 40, 16, 4
    starts = [np.concatenate([[0], np.cumsum(n)]) for n in (r.integers(0, 28, B), np.eye(B, dtype=int)[60] * 1200 + r.integers(0, 3, B))]
    start = torch.tensor(starts[0], dtype=torch.int32, device="cuda")
    d, c = Scan(r, B, 0, C, N, 1, "bf16", packed_rows=T), Conv(r, B, 0, C, W, "bf16", packed_rows=T)
    st = status()
    kw = dict(seq_start=start, status_dev=st)
    sf, sb, cf, cb = A.make_scan_cfg(B, T, C, N, **kw), A.make_scan_cfg(B, T, C, N, **kw), A.make_conv_cfg(B, T, C, W, **kw), A.make_conv_cfg(B, T, C, W, **kw)
    space(sf, A.atlas_scan_workspace_bytes(sf))
    space(sb, A.atlas_scan_backward_workspace_bytes(sb))
    space(cb, A.atlas_conv_backward_workspace_bytes(cb))
    o = d.grads()
    o.update(y=torch.zeros_like(d.x), h=d.h.clone(), dh=d.dh.clone(), cy=torch.zeros_like(c.x), cs=c.s.clone(), cdx=torch.zeros_like(c.x), cds=c.ds.clone(),
             cdw=torch.zeros(C, W, device="cuda"), cdb=torch.zeros(C, device="cuda"))

    def everything():
        o["dh"].copy_(d.dh)
        o["cds"].copy_(c.ds)
        A.atlas_scan_forward(*d.inputs(), sf, o["y"], d.h, o["h"])
        A.atlas_scan_backward(*d.inputs(), sb, d.h, d.dy, o["dh"], o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], o["dD"], o["dz"], o["ddt_bias"])
        A.atlas_conv_forward(c.x, c.w, c.b, cf, o["cy"], c.s, o["cs"])
        A.atlas_conv_backward(c.x, c.w, c.b, cb, c.s, c.dy, o["cds"], o["cdx"], o["cdw"], o["cdb"])
    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        everything()
    for s in starts[::-1]:
        start.copy_(torch.from_numpy(s))
        for v in o.values():
            v.zero_()
        everything()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in o.items()}
        for v in o.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], o[k]) for k in o) and int(st) == 0
    for b in (0, 59, 60, 99):
        rows = slice(starts[0][b], starts[0][b + 1])
        d.check(o["y"][rows], o["h"][b], rows, d.h_h[b], f"sequence {b}")
        c.check(o["cy"][rows], o["cs"][b], rows, c.sh[b], "bf16", f"sequence {b}")
