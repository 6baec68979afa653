"""The gated linear recurrence on the GPU against the 64-bit reference of more_ops_ref.py: types, odd widths, lengths
from none to several groups of tiles, packed sequences, slots with padding, extreme gates, strides, streams and
captured graphs, gradients, and a layer of it between norm and convolution.  Tolerances: see more_ops_ref.py."""
import numpy as np
import pytest

import more_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_layer_ops import CODE, DT, LENS, TYPES, _lib, close, dev, draw, host, packed, rng, space, status  # noqa: E402,F401

pytestmark = pytest.mark.gpu
C = 8.0


class Glr:
    """One call's data on both sides."""

    def __init__(self, r, B, L, D, dtype, gate=True, inp=True, bias=True, n=None, packed_rows=None, slow=False):
        lead = (packed_rows,) if packed_rows else (B, L)
        self.x, self.xh = draw(r, (*lead, D), dtype)
        self.r, self.rh = draw(r, (*lead, D), dtype)
        self.i, self.ih = draw(r, (*lead, D), dtype) if inp else (None, None)
        self.z, self.zh = draw(r, (*lead, D), dtype) if gate else (None, None)
        self.lam = dev(r.uniform(-6, -4, D) if slow else r.uniform(-6, 1, D))
        self.lamh = host(self.lam)
        self.rb, self.rbh = draw(r, D, "fp32", 0.3) if bias else (None, None)
        self.ib, self.ibh = draw(r, D, "fp32", 0.3) if bias and inp else (None, None)
        self.h, self.hh = draw(r, (n or B, D), "fp32")
        self.dtype, self.D = dtype, D

    def ref(self, at, h0, *grads, mag=False):
        """at: indexes a sequence's rows"""
        z, i = (None if t is None else t[at] for t in (self.zh, self.ih))
        return R.glr(self.xh[at], self.rh[at], i, z, self.lamh, self.rbh, self.ibh, C, h0, *grads, mag=mag)

    def cfg(self, B, L, **kw):
        cfg = A.make_glr_cfg(B, L, self.D, c=C, dtype=CODE[self.dtype], **kw)
        space(cfg, max(A.atlas_glr_workspace_bytes(cfg), 0 if cfg.slot else A.atlas_glr_backward_workspace_bytes(cfg)))
        return cfg

    def forward(self, cfg, y, h_out=None, kept=None, h_in="own"):
        A.atlas_glr_forward(self.x, self.r, self.i, self.z, self.lam, self.rb, self.ib, cfg, y, self.h if h_in == "own" else h_in, h_out, kept)

    def backward(self, cfg, dy, dh, kept=None):
        o = {k: torch.full_like(t, 7.0) for k, t in (("dx", self.x), ("dr", self.r), ("di", self.i), ("dz", self.z), ("dlam", self.lam),
                                                    ("drb", self.rb), ("dib", self.ib)) if t is not None}
        A.atlas_glr_backward(self.x, self.r, self.i, self.z, self.lam, self.rb, self.ib, cfg, self.h, kept, dy, dh, o["dx"], o["dr"],
                             o.get("di"), o.get("dz"), o["dlam"], o.get("drb"), o.get("dib"))
        return o


def kept_of(cfg):
    return torch.full((A.atlas_glr_kept_bytes(cfg),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate,inp,bias", [(True, True, True), (False, False, False)])
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (3, 1, 37), (2, 1, 520), (1, 2, 32), (2, 5, 7), (3, 127, 33), (2, 128, 64), (2, 129, 36), (1, 2049, 40),
                                   (3, 2176, 12), (1, 4500, 35), (200, 3, 8)])
def test_forward(B, L, D, gate, inp, bias, dtype):
    g = Glr(rng(50, B, L, D), B, L, D, dtype, gate, inp, bias)
    cfg = g.cfg(B, L)
    y, out = torch.full_like(g.x, 5.0), torch.full_like(g.h, 5.0)
    g.forward(cfg, y, out)
    zero = torch.full_like(g.x, 5.0)
    g.forward(cfg, zero, None, h_in=None)
    for b in range(min(B, 4)):
        for got, h0 in ((y, g.hh[b]), (zero, np.zeros(D))):
            ref, S = g.ref(b, h0), g.ref(b, h0, mag=True)
            close(got[b], ref["y"], S["y"], dtype, L, "y")
        ref, S = g.ref(b, g.hh[b]), g.ref(b, g.hh[b], mag=True)
        close(out[b], ref["h"], S["h"], "fp32", L, "h")


def check_grads(g, o, dh, seqs, dyh, dhh, carry=None):
    """seqs: (index of a sequence's rows, its number)"""
    sums = {k: [np.zeros(g.D), np.zeros(g.D)] for k in ("dlam", "drb", "dib")}
    longest = 1
    for at, b, n in seqs:
        h0 = g.hh[b] * (1 if carry is None else carry[b])
        args = (dyh[at], dhh[b])
        ref, S = g.ref(at, h0, *args), g.ref(at, h0, *args, mag=True)
        longest = max(longest, n)
        for k in ("dx", "dr", "di", "dz"):
            if k in o:
                close(o[k][at], ref[k], S[k], g.dtype, n, k)
        if dh is not None:
            keep = 1 if carry is None else carry[b]
            close(dh[b], ref["dh"] * keep, S["dh"], "fp32", n, "dh")
        for k in sums:
            if k in ref:
                sums[k][0] += ref[k]
                sums[k][1] += S[k]
    for k in sums:
        if k in o:
            close(o[k], *sums[k], "fp32", longest + sum(n for *_, n in seqs) / 32, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate,inp,bias,keep", [(True, True, True, True), (False, False, False, False)])
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (3, 1, 37), (1, 2, 32), (2, 5, 7), (3, 127, 33), (2, 128, 64), (2, 129, 36), (1, 2049, 40), (3, 2176, 12),
                                   (1, 4500, 35), (200, 3, 8)])
def test_backward(B, L, D, gate, inp, bias, keep, dtype):
    r = rng(51, B, L, D)
    g = Glr(r, B, L, D, dtype, gate, inp, bias)
    (dy, dyh), (dh, dhh) = draw(r, (B, L, D), dtype), draw(r, (B, D), "fp32")
    cfg = g.cfg(B, L)
    kept = None
    if keep:
        kept = kept_of(cfg)
        g.forward(cfg, torch.empty_like(g.x), None, kept)
    o = g.backward(cfg, dy, dh, kept)
    check_grads(g, o, dh, [(b, b, L) for b in range(B)], dyh, dhh)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", LENS + [[128, 0, 128, 1], [2048, 2048], [0, 0, 0], [3] * 300], ids=lambda v: str(len(v)) + "x" + str(max(v)))
@pytest.mark.parametrize("D,front", [(36, 0), (33, 130)])
def test_packed(lens, D, front, dtype):
    """Empty sequences pass their states on; rows in front of the first and behind the last stay."""
    r = rng(52, len(lens), D)
    start, rows, at = packed(lens, 5, front)
    B = len(lens)
    g = Glr(r, B, 0, D, dtype, packed_rows=rows, n=B + 2)
    carry = torch.tensor([b % 3 != 1 for b in range(B)], dtype=torch.uint8, device="cuda")
    slot = torch.tensor([(b + 2) % (B + 2) if b % 5 != 4 else -1 for b in range(B)], dtype=torch.int32, device="cuda")
    st = status()
    for x in (g.x, g.r, g.i, g.z):  # nothing of the rows around is read into anything
        x[:front], x[at[-1]:] = float("nan"), float("nan")
    cfg = g.cfg(B, rows, seq_start=start, slot=slot, n_slots=B + 2, carry=carry, status_dev=st)
    y, pool = torch.full_like(g.x, 5.0), g.h.clone()
    A.atlas_glr_forward(g.x, g.r, g.i, g.z, g.lam, g.rb, g.ib, cfg, y, pool, pool)
    assert int(st) == 0
    left = np.ones(rows, bool)
    used = set()
    for b, n in enumerate(lens):
        if b % 5 == 4:
            continue
        k = (b + 2) % (B + 2)
        used.add(k)
        rows_b = slice(at[b], at[b] + n)
        left[rows_b] = False
        h0 = g.hh[k] * (b % 3 != 1)
        ref, S = g.ref(rows_b, h0), g.ref(rows_b, h0, mag=True)
        close(y[rows_b], ref["y"], S["y"], dtype, n, "y")
        close(pool[k], ref["h"], S["h"], "fp32", n, "h")
    assert (y[torch.from_numpy(left).cuda()] == 5).all()
    for k in range(B + 2):
        if k not in used:
            assert torch.equal(pool[k], g.h[k])
    # backward: states by number
    cfg = g.cfg(B, rows, seq_start=start, carry=carry, status_dev=st)
    (dy, dyh), (dh, dhh) = draw(r, (rows, D), dtype), draw(r, (B, D), "fp32")
    kept = kept_of(cfg)
    g.forward(cfg, torch.empty_like(g.x), None, kept)
    grads, again = dh.clone(), dh.clone()
    o, o2 = g.backward(cfg, dy, grads, kept), g.backward(cfg, dy, again)
    for k in o:
        assert torch.equal(o[k], o2[k]), k
    assert torch.equal(grads, again) and int(st) == 0
    check_grads(g, o, grads, [(slice(at[b], at[b] + n), b, n) for b, n in enumerate(lens)], dyh, dhh, [b % 3 != 1 for b in range(B)])
    around = np.ones(rows, bool)
    around[at[0]:at[-1]] = False
    for k in ("dx", "dr", "di", "dz"):
        assert (o[k][torch.from_numpy(around).cuda()] == 7).all(), k


@pytest.mark.parametrize("bad", ["falls", "beyond", "negative", "slot", "twice"])
def test_bad_sequences_are_left_out_and_reported(bad):
    D, rows = 40, 300
    start = [0, 100, 200, 300]
    slot = [0, 1, 2]
    good = [True, True, True]
    if bad == "falls":
        start, good = [0, 100, 50, 300], [True, False, False]
    if bad == "beyond":
        start, good = [0, 100, 200, 301], [True, True, False]
    if bad == "negative":
        start, good = [-1, 100, 200, 300], [False, True, True]
    if bad == "slot":
        slot, good = [0, 5, 2], [True, False, True]
    if bad == "twice":
        slot, good = [0, 1, 1], [True, True, False]
    g = Glr(rng(53), 3, 0, D, "fp32", packed_rows=rows, n=3)
    st = status()
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cfg = g.cfg(3, rows, seq_start=as_int(start), slot=as_int(slot), n_slots=3, status_dev=st)
    y, out = torch.full_like(g.x, 5.0), torch.full_like(g.h, 5.0)
    g.forward(cfg, y, out)
    assert int(st) == A.ERR_INVALID
    for b in range(3):
        if good[b]:
            at = slice(start[b], start[b + 1])
            ref, S = g.ref(at, g.hh[slot[b]]), g.ref(at, g.hh[slot[b]], mag=True)
            close(y[at], ref["y"], S["y"], "fp32", rows, "y")
            close(out[slot[b]], ref["h"], S["h"], "fp32", rows, "h")
        elif bad in ("slot", "twice", "beyond"):
            assert (y[start[b]:min(start[b + 1], rows)] == 5).all()
    if bad in ("falls", "beyond", "negative"):
        o = g.backward(g.cfg(3, rows, seq_start=as_int(start), status_dev=st), torch.ones_like(g.x), None)
        torch.cuda.synchronize()
        assert o["dx"].shape == g.x.shape and int(st) == A.ERR_INVALID


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8, 37])
def test_tokens_continue_a_prompt(D, dtype):
    """A prompt in one call, and its first part in a call and the rest token by token from slots in another order."""
    B, L, cut = 5, 140, 133
    g = Glr(rng(54, D), B, L, D, dtype)
    y, end = torch.empty_like(g.x), torch.empty_like(g.h)
    g.forward(g.cfg(B, L), y, end)
    part = lambda t, s: None if t is None else t[:, s].contiguous()  # noqa: E731
    pool = torch.full((9, D), 3.0, device="cuda")
    at = [7, 0, 4, 2, 8]
    head = [part(t, slice(0, cut)) for t in (g.x, g.r, g.i, g.z)]
    slot = torch.tensor(at, dtype=torch.int32, device="cuda")
    pool[slot.long()] = g.h
    cfg = g.cfg(B, cut, slot=slot, n_slots=9)
    y0 = torch.empty_like(head[0])
    A.atlas_glr_forward(*head, g.lam, g.rb, g.ib, cfg, y0, pool, pool)
    for b in range(B):  # (its tiles begin at other rows: other orders of the same sums)
        ref, S = g.ref((b, slice(0, cut)), g.hh[b]), g.ref((b, slice(0, cut)), g.hh[b], mag=True)
        close(y0[b], ref["y"], S["y"], dtype, cut, "head")
    step = g.cfg(B + 1, 1, slot=torch.tensor(at + [-1], dtype=torch.int32, device="cuda"), n_slots=9)
    for t in range(cut, L):
        one = [torch.cat([v[:, t], torch.full((1, D), float("nan"), device="cuda", dtype=v.dtype)]) for v in (g.x, g.r, g.i, g.z)]
        yt = torch.full((B + 1, D), 5.0, device="cuda", dtype=DT[dtype])
        A.atlas_glr_forward(*one, g.lam, g.rb, g.ib, step, yt, pool, pool)
        S = np.abs(host(y[:, t])) + 1
        close(yt[:B], host(y[:, t]), S, dtype, 2 * L, "token")
        assert (yt[B] == 5).all()
    close(pool[slot.long()], host(end), np.abs(host(end)) + 1, "fp32", 2 * L, "state")
    assert (pool[[1, 3, 5, 6]] == 3).all()


@pytest.mark.parametrize("D", [8, 33])
def test_extreme_gates(D):
    """Closed and open gates, a rate of nothing and a large one: no NaN, no lost state."""
    L = 260
    g = Glr(rng(55, D), 1, L, D, "fp32", bias=False)
    r, i = np.zeros((L, D)), np.zeros((L, D))
    lam = np.resize([-200.0, -90.0, -30.0, 0.0, 30.0, 200.0, 1e30], D)
    r[:, 0::5], r[:, 1::5], r[:, 2::5], r[:, 3::5] = -300, 300, -40, -np.inf
    i[::3], i[1::3] = -300, 300
    g.r, g.i, g.lam = dev(r[None]), dev(i[None]), dev(lam)
    y, out = torch.empty_like(g.x), torch.empty_like(g.h)
    cfg = g.cfg(1, L)
    kept = kept_of(cfg)
    g.forward(cfg, y, out, kept)
    with np.errstate(over="ignore", under="ignore"):
        lamh = host(g.lam)
        args = (g.xh[0], np.maximum(r, -700), np.maximum(i, -700), g.zh[0], lamh, None, None, C, g.hh[0])
        ref, S = R.glr(*args), R.glr(*args, mag=True)
        dy, dh = draw(rng(56, D), (1, L, D), "fp32"), draw(rng(57, D), (1, D), "fp32")
        grads = R.glr(*args, dy[1][0], dh[1][0]), R.glr(*args, dy[1][0], dh[1][0], mag=True)
    close(y[0], ref["y"], S["y"], "fp32", L, "y")
    close(out[0], ref["h"], S["h"], "fp32", L, "h")
    state = dh[0].clone()
    o = g.backward(cfg, dy[0], state, kept)
    for k in ("dx", "dr", "di", "dz"):
        # gates below 2^-120 are held there: what they let through is at most sqrt(2^-120) of a term of 1
        close(o[k][0], grads[0][k], grads[1][k] + 2.0 ** -38, "fp32", L, k)
    close(state[0], grads[0]["dh"], grads[1]["dh"], "fp32", L, "dh")
    for k in ("dlam", "drb", "dib"):
        if k in o:
            close(o[k], grads[0][k], grads[1][k] + 2.0 ** -38, "fp32", L, k)


@pytest.mark.parametrize("dtype", TYPES)
def test_gates_of_the_lowest_value(dtype):
    """Output and input gates of the type's lowest and largest number: outputs and gradients of 0 where the gate is
    closed, as of a token that is masked, and none that are not finite."""
    L, D = 200, 40
    low, high = -float(torch.finfo(DT[dtype]).max), 40.0
    g = Glr(rng(68), 1, L, D, dtype)
    g.z[:, ::2], g.i[:, ::3], g.r[:, ::5] = low, low, low
    g.z[:, 1::4], g.r[:, 1::5] = high, high
    dy, dh = torch.ones_like(g.x), torch.ones_like(g.h)
    cfg = g.cfg(1, L)
    y = torch.empty_like(g.x)
    g.forward(cfg, y)
    o = g.backward(cfg, dy, dh)
    for t in (y, *o.values()):
        assert torch.isfinite(t).all()
    assert not y[:, ::2].any() and not o["dz"][:, ::2].any()
    assert not o["di"][:, ::3].any() and not o["dr"][:, ::5].any()
    assert o["dz"][:, 1::4].any()


def test_a_slow_channel_over_many_tokens():
    """Decays of 1 - 1e-4 .. 1 - 1e-6 over 40000 tokens: the rounding of a does not add up to a drift.  u keeps its
    relative precision there (1 - a^2 of a rounded a would be off by up to 2^-25 / 1e-6)."""
    L, D = 40000, 32
    r = rng(58)
    g = Glr(r, 1, L, D, "fp32", gate=False, inp=False, bias=False)
    g.lam = dev(np.log(np.expm1(10.0 ** r.uniform(-6, -4, D) / C * 2)))
    g.lamh = host(g.lam)
    g.x = g.x.abs()
    g.xh = np.abs(g.xh)
    y, out = torch.empty_like(g.x), torch.empty_like(g.h)
    g.forward(g.cfg(1, L), y, out)
    ref = g.ref(0, g.hh[0])
    # roundings of a: 2^-25 a step of either sign, so sqrt(L) 2^-25 and not L 2^-25, six deviations wide
    assert (np.abs(host(out[0]) - ref["h"]) <= 6 * L ** 0.5 * 2.0 ** -25 * np.abs(ref["h"]) + 2.0 ** -20 * np.abs(ref["h"])).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("extra,shift", [(4, 0), (3, 0), (4, 1)])
def test_strides_and_order(extra, shift, dtype):
    """Tokens in front of batches, gaps between rows, addresses off a boundary; gradients with their inputs' strides."""
    B, L, D = 3, 150, 36
    r = rng(59, extra, shift)
    g = Glr(r, B, L, D, dtype)
    (dy, dyh), (dh, dhh) = draw(r, (B, L, D), dtype), draw(r, (B, D), "fp32")

    def laid(t, tokens_first):
        w = D + extra
        buf = torch.full((B * L * w + shift,), 7.0, device="cuda", dtype=DT[dtype])
        s = (w, B * w) if tokens_first else (L * w, w)
        v = buf[shift:].as_strided((B, L, D), (*s, 1))
        v.copy_(t) if t is not None else None
        return v, s, buf
    x, sx, _ = laid(g.x, True)
    rr, sr, _ = laid(g.r, False)
    z, sz, _ = laid(g.z, True)
    y, sy, buf = laid(None, True)
    kw = dict(x_strides=sx, r_strides=sr, z_strides=sz, y_strides=sy)
    cfg = g.cfg(B, L, **kw)
    flat = lambda v: v.as_strided((v.untyped_storage().nbytes() // v.element_size() - v.storage_offset(),), (1,))  # noqa: E731
    A.atlas_glr_forward(flat(x), flat(rr), g.i, flat(z), g.lam, g.rb, g.ib, cfg, flat(y), g.h)
    plain = torch.empty_like(g.x)
    g.forward(g.cfg(B, L), plain)
    for b in range(B):
        close(y[b], g.ref(b, g.hh[b])["y"], g.ref(b, g.hh[b], mag=True)["y"], dtype, L, "y")
    assert int((buf != 7).sum()) <= B * L * D
    outs = {k: laid(None, f) for k, f in (("dx", True), ("dr", False), ("dz", True))}
    di, dlam, drb, dib = torch.empty_like(g.i), *(torch.empty(D, device="cuda") for _ in range(3))
    up, _, _ = laid(dy, True)
    A.atlas_glr_backward(flat(x), flat(rr), g.i, flat(z), g.lam, g.rb, g.ib, cfg, g.h, None, flat(up), dh, flat(outs["dx"][0]), flat(outs["dr"][0]),
                         di, flat(outs["dz"][0]), dlam, drb, dib)
    o = dict(dx=outs["dx"][0], dr=outs["dr"][0], dz=outs["dz"][0], di=di, dlam=dlam, drb=drb, dib=dib)
    check_grads(g, o, dh, [(b, b, L) for b in range(B)], dyh, dhh)


def test_gradients_are_the_differences():
    """The kernels' gradients along a direction of length 1 against differences of the kernels' own outputs in 32 bits."""
    B, L, D, step = 2, 150, 12, 2.0 ** -5
    r = rng(60)
    g = Glr(r, B, L, D, "fp32")
    dy, dh = draw(r, (B, L, D), "fp32")[0], draw(r, (B, D), "fp32")[0]
    cfg = g.cfg(B, L)
    back = dh.clone()
    o = g.backward(cfg, dy, back)
    o["dh0"] = back

    def loss():
        y, h = torch.empty_like(g.x), torch.empty_like(g.h)
        g.forward(cfg, y, h)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())
    for name, k in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("lam", "dlam"), ("rb", "drb"), ("ib", "dib"), ("h", "dh0")):
        v = getattr(g, name)
        u = draw(r, v.shape, "fp32")[0]
        u /= u.norm()
        ends = []
        for sign in (1, -1):
            setattr(g, name, v + sign * step * u)
            ends.append(loss())
        setattr(g, name, v)
        want = float((o[k].double() * u.double()).sum())
        assert abs((ends[0] - ends[1]) / (2 * step) - want) < 2e-3 * (1 + float(o[k].norm())), name


def test_equal_bits_and_captured_graphs():
    """Equal calls give equal bits; two captured training passes with a workspace each, replayed together on two
    streams, and again on other starts, give those of eager calls."""
    r = rng(61)
    B, rows, D = 4, 9000, 130
    g = Glr(r, B, 0, D, "bf16", packed_rows=rows)
    dy, dh0 = draw(r, (rows, D), "bf16")[0], draw(r, (B, D), "fp32")[0]
    starts = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 3000, 3000, 8990, 9000], [5, 100, 4000, 4001, 8999])]

    def plan():
        start, dh, y, h = starts[0].clone(), dh0.clone(), torch.zeros_like(g.x), torch.zeros_like(g.h)
        cfg = g.cfg(B, rows, seq_start=start)
        o = {k: torch.zeros_like(t) for k, t in (("dx", g.x), ("dr", g.r), ("di", g.i), ("dz", g.z), ("dlam", g.lam), ("drb", g.rb), ("dib", g.ib))}
        kept = kept_of(cfg)

        def call():
            dh.copy_(dh0)
            g.forward(cfg, y, h, kept)
            A.atlas_glr_backward(g.x, g.r, g.i, g.z, g.lam, g.rb, g.ib, cfg, g.h, kept, dy, dh, *o.values())
        return call, start, [dh, y, h, *o.values()]
    want = []
    for s in starts:
        call, start, outs = plan()
        start.copy_(s)
        call()
        first = [t.clone() for t in outs]
        call()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        want.append(first)
    graphs = []
    for _ in range(2):
        call, start, outs = plan()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            call()
        graphs.append((graph, stream, start, outs))
    for turn in (0, 1, 0):
        for graph, stream, start, outs in graphs:
            start.copy_(starts[turn])
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for graph, stream, start, outs in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for *_, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want[turn], outs))


def test_no_rows_pass_states_on():
    g = Glr(rng(62), 3, 0, 40, "fp32")
    cfg = g.cfg(3, 0, carry=torch.tensor([1, 0, 1], dtype=torch.uint8, device="cuda"))
    out = torch.full_like(g.h, 5.0)
    g.forward(cfg, None, out)
    assert torch.equal(out[[0, 2]], g.h[[0, 2]]) and not out[1].any()
    dh = g.h.clone()
    dlam, drb, dib = (torch.full((40,), 5.0, device="cuda") for _ in range(3))
    A.atlas_glr_backward(None, None, g.i, None, g.lam, g.rb, g.ib, cfg, g.h, None, None, dh, None, None, g.i, None, dlam, drb, dib)
    assert torch.equal(dh[[0, 2]], g.h[[0, 2]]) and not dh[1].any() and not (dlam.any() or drb.any() or dib.any())


def test_rows_past_32_bits():
    """More than 2^32 elements in a tensor: the last sequence is as it is alone."""
    B, L, D = 33, 65600, 2048
    r = rng(63)
    t = {k: torch.zeros(B, L, D, dtype=torch.bfloat16, device="cuda") for k in ("x", "r")}
    for k in t:
        t[k][-1] = torch.from_numpy(r.standard_normal((L, D)).astype(np.float32)).cuda()
    lam, h0 = dev(r.uniform(-6, -4, D)), dev(r.standard_normal((B, D)))
    outs = []
    for n in (B, 1):
        cfg = A.make_glr_cfg(n, L, D, c=C)
        space(cfg, A.atlas_glr_workspace_bytes(cfg))
        y, h = torch.empty(n, L, D, dtype=torch.bfloat16, device="cuda"), torch.empty(n, D, device="cuda")
        A.atlas_glr_forward(t["x"][-n:], t["r"][-n:], None, None, lam, None, None, cfg, y, h0[-n:].contiguous(), h)
        outs.append((y[-1].clone(), h[-1].clone()))
        del y
    (y, h), (y1, h1) = outs
    # the sequences' tiles begin elsewhere: other orders of the same sums
    assert (h - h1).abs().max() <= 2.0 ** -14 * h1.abs().max()
    assert (y.float() - y1.float()).abs().max() <= 2.0 ** -6 * y1.float().abs().max() and y1.float().abs().max() > 0.1


def test_tensors_are_checked():
    B, L, D = 2, 5, 8
    g = Glr(rng(64), B, L, D, "bf16")
    cfg = g.cfg(B, L)
    y, kept = torch.empty_like(g.x), kept_of(cfg)
    args = dict(x=g.x, r=g.r, i=g.i, z=g.z, lam=g.lam, rb=g.rb, ib=g.ib, y=y, h=g.h, out=g.h, kept=kept)

    def call(**kw):
        u = {**args, **kw}
        A.atlas_glr_forward(u["x"], u["r"], u["i"], u["z"], u["lam"], u["rb"], u["ib"], cfg, u["y"], u["h"], u["out"], u["kept"])
    call()
    for k, bad in (("x", g.x.float()), ("r", g.r[:1]), ("i", g.i.cpu()), ("z", g.z[:, :4]), ("lam", g.lam.bfloat16()), ("rb", g.rb[:4]), ("ib", g.ib.double()),
                   ("y", y[:1]), ("h", g.h[:1]), ("out", g.h.bfloat16()), ("kept", kept[:8]), ("kept", kept.cpu()), ("h", g.h.t().contiguous().t())):
        with pytest.raises(A.AtlasError):
            call(**{k: bad})


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [40, 33])
@pytest.mark.parametrize("lens", [[5, 7, 6], [300, 129, 700, 2], [128, 128, 128], [5000, 40, 5000]], ids=str)
def test_what_is_not_finite_stays_in_its_sequence(lens, D, dtype):
    """The second sequence has NaN inputs and gates and an infinite state: the others' outputs and gradients are, bit by
    bit, those beside a finite one."""
    r = rng(66, len(lens), D)
    start, rows, at = packed(lens, 0)
    B = len(lens)
    g = Glr(r, B, 0, D, dtype, packed_rows=rows)
    dy, dh0 = draw(r, (rows, D), dtype)[0], draw(r, (B, D), "fp32")[0]
    cfg = g.cfg(B, rows, seq_start=start)

    def run():
        y, h, dh, kept = torch.zeros_like(g.x), torch.zeros_like(g.h), dh0.clone(), kept_of(cfg)
        g.forward(cfg, y, h, kept)
        o = g.backward(cfg, dy, dh, kept)
        return [y, o["dx"], o["dr"], o["di"], o["dz"]], [h, dh]
    want = run()
    mid = slice(at[1], at[2])
    g.x[mid], g.h[1] = float("nan"), float("inf")
    g.r[mid.start + 1:mid.stop] = float("nan")
    dy[mid], dh0[1] = float("inf"), float("nan")
    got = run()
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[mid] = False
    for a, b in zip(got[0], want[0]):
        assert torch.equal(a[others], b[others])
        assert not torch.isfinite(a[mid].float()).all()
    for a, b in zip(got[1], want[1]):
        assert torch.equal(a[[b for b in range(B) if b != 1]], b[[b for b in range(B) if b != 1]])


def test_a_tile_that_is_lost_ends_the_waits_and_is_reported():
    """A separately built copy of the library in which the second tile of the first 32 channels never hands on its map: the
    wait for it runs out, the others give up at once, the status word says so, the other channels are right, and the
    next call is."""
    import time

    from test_memorization_recurrent_gb300 import build
    lib = A.open_library(build.build_variant("atlasmem_withhold", ["ATLAS_TEST_WITHHOLD_LOADS"]))
    L, D = 128 * 40, 40
    g = Glr(rng(67), 1, L, D, "fp32")
    st = status()
    cfg = g.cfg(1, L, status_dev=st)
    want, y = torch.empty_like(g.x), torch.zeros_like(g.x)
    g.forward(cfg, want)
    torch.cuda.synchronize()
    begin = time.monotonic()
    p = lambda t: t.data_ptr()  # noqa: E731
    assert lib.atlas_glr_forward(p(g.x), p(g.r), p(g.i), p(g.z), p(g.lam), p(g.rb), p(g.ib), cfg, p(y), p(g.h), None, None,
                                 torch.cuda.current_stream().cuda_stream) == A.OK
    torch.cuda.synchronize()
    assert time.monotonic() - begin < 30
    assert int(st) == A.ERR_TIMEOUT
    assert torch.equal(y[..., 32:], want[..., 32:]) and torch.equal(y[:, :256], want[:, :256])
    assert torch.isnan(y[:, 256:384, :32]).all()
    st.zero_()
    g.forward(cfg, y)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(y, want)


def test_a_layer_of_them():
    """Layer norm, short convolution, gated linear recurrence and a residual layer norm, forward and backward through
    each, against differences along directions of the input and of parameters (in 32 bits)."""
    B, L, D, W, step = 2, 70, 24, 4, 2.0 ** -5
    r = rng(65)
    p = {k: draw(r, s, "fp32", f)[0] for k, s, f in (("x", (B, L, D), 1), ("w1", D, 1), ("b1", D, 0.3), ("taps", (D, W), 0.5), ("wr", (D, D), 0.2),
                                                      ("wi", (D, D), 0.2), ("lam", D, 0.5), ("w2", D, 1), ("b2", D, 0.3))}
    dout = draw(r, (B, L, D), "fp32")[0]
    norm = A.make_norm_cfg(B * L, D, dtype=A.F32, eps=1e-5)
    conv, glr = A.make_conv_cfg(B, L, D, W, dtype=A.F32), A.make_glr_cfg(B, L, D, c=C, dtype=A.F32)
    space(norm, A.atlas_layernorm_backward_workspace_bytes(norm))
    space(conv, A.atlas_conv_backward_workspace_bytes(conv))
    space(glr, max(A.atlas_glr_workspace_bytes(glr), A.atlas_glr_backward_workspace_bytes(glr)))
    kept = kept_of(glr)
    new = lambda: torch.empty(B, L, D, device="cuda")  # noqa: E731

    def forward(p):
        n1, cv, y, out, res = (new() for _ in range(5))
        A.atlas_layernorm_forward(p["x"], None, p["w1"], p["b1"], norm, n1)
        A.atlas_conv_forward(n1, p["taps"], None, conv, cv)
        rr, ii = cv @ p["wr"], cv @ p["wi"]
        A.atlas_glr_forward(cv, rr, ii, n1, p["lam"], None, None, glr, y, None, None, kept)
        A.atlas_layernorm_forward(y, p["x"], p["w2"], p["b2"], norm, out, res)
        return n1, cv, rr, ii, y, out, res

    def loss(p):
        return float((forward(p)[5].double() * dout.double()).sum())
    n1, cv, rr, ii, y, out, res = forward(p)
    g, small = {}, lambda: torch.empty(D, device="cuda")
    dres, g["w2"], g["b2"] = new(), small(), small()
    A.atlas_layernorm_backward(res, p["w2"], dout, None, norm, dres, g["w2"], g["b2"])
    dcv, drr, dii, dn1, g["lam"] = new(), new(), new(), new(), small()
    A.atlas_glr_backward(cv, rr, ii, n1, p["lam"], None, None, glr, None, kept, dres, None, dcv, drr, dii, dn1, g["lam"], None, None)
    g["wr"], g["wi"] = (cv.flatten(0, 1).T @ d.flatten(0, 1) for d in (drr, dii))
    dcv += drr @ p["wr"].T + dii @ p["wi"].T
    dc, g["taps"] = new(), torch.empty(D, W, device="cuda")
    A.atlas_conv_backward(n1, p["taps"], None, conv, None, dcv, None, dc, g["taps"], None)
    g["x"], g["w1"], g["b1"] = new(), small(), small()
    A.atlas_layernorm_backward(p["x"], p["w1"], dc + dn1, dres, norm, g["x"], g["w1"], g["b1"])
    for k in g:
        u = draw(r, p[k].shape, "fp32")[0]
        u /= u.norm()
        diff = (loss({**p, k: p[k] + step * u}) - loss({**p, k: p[k] - step * u})) / (2 * step)
        assert abs(diff - float((g[k].double() * u.double()).sum())) < 5e-3 * (1 + float(g[k].norm())), k
