"""The operators of a recurrent layer around the memory update, as cases to time and compare.

Three operators, forward and backward, for prompts and for single tokens:

norm  residual addition and root-mean-square norm, with a bf16 / fp16 / fp32 output or e4m3
      with one scale per row or per group of channels
conv  short causal convolution per channel with SiLU, its last inputs carried as a state
scan  selective state space scan  h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t,  y_t = C_t h_t + D x_t,
      gated by SiLU(z), its state carried

`run` computes them in plain torch operations, or (own = True) through this repository's entry
points.  The largest cases have the tokens and the width of the DeltaNet-like workload
(8 sequences x 4096 tokens, 16 heads x 128).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # the tokens of one decoding step entering a layer whose projections take 8 bits
        dict(name="norm-token", op="norm", rows=8, d=2048, dtype="bf16", r_dtype="bf16", out="e4m3", group=0, residual=True),
        # every token of the prompts entering a layer, scales per 128 channels
        dict(name="norm-prompt", op="norm", rows=32768, d=2048, dtype="bf16", r_dtype="bf16", out="e4m3", group=128, residual=True),
        # the keys of all heads and tokens, each normalised over its 128 channels
        dict(name="norm-keys", op="norm", rows=524288, d=128, dtype="bf16", r_dtype="bf16", out="bf16", group=0, residual=False),
        # the training pass of a norm with a residual stream held in 32 bits
        dict(name="norm-train", op="norm_bwd", rows=16384, d=2560, dtype="bf16", r_dtype="fp32", residual=True),
        # one decoding step of 64 sequences whose states lie in a larger pool
        dict(name="conv-token", op="conv", B=64, L=1, C=2048, W=4, dtype="bf16", act=True, head_dim=0, slots=96, ragged=0),
        # prompts: the convolution in front of the memory, written head by head as the memory reads it
        dict(name="conv-prompt", op="conv", B=8, L=4096, C=2048, W=4, dtype="bf16", act=True, head_dim=128, slots=0, ragged=0),
        # a packed batch of prompts of unequal lengths, odd width, with states carried on
        dict(name="conv-packed", op="conv", B=11, L=9001, C=1500, W=4, dtype="fp16", act=True, head_dim=0, slots=16, ragged=5),
        # its training pass
        dict(name="conv-train", op="conv_bwd", B=8, L=4096, C=2048, W=4, dtype="bf16", act=True, head_dim=0, slots=0, ragged=0),
        # one decoding step of 64 sequences
        dict(name="scan-token", op="scan", B=64, L=1, D=2048, N=16, G=1, dtype="bf16", gate=True, slots=96, ragged=0),
        # prompts
        dict(name="scan-prompt", op="scan", B=8, L=4096, D=2048, N=16, G=1, dtype="bf16", gate=True, slots=0, ragged=0),
        # a few long prompts packed into one row: little parallel work but the length
        dict(name="scan-packed", op="scan", B=3, L=16384, D=1024, N=16, G=1, dtype="bf16", gate=True, slots=4, ragged=7),
        # the training pass
        dict(name="scan-train", op="scan_bwd", B=4, L=2048, D=2048, N=16, G=1, dtype="bf16", gate=True, slots=0, ragged=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "conv", "conv", "conv_bwd", "scan", "scan", "scan_bwd"])
    if op.startswith("norm"):
        d = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            d = max(16, d // 16 * 16)
        rows = _log(rng, 1, max(2, min(524288, 32768 * 2048 // d)))
        c = dict(op=op, rows=rows, d=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        c["r_dtype"] = rng.choice([c["dtype"], "fp32"])
        c["residual"] = rng.random() < 0.7
        if not c["residual"]:
            c["r_dtype"] = c["dtype"]
        if op == "norm":
            c["out"] = rng.choice([c["dtype"], "e4m3"])
            c["group"] = rng.choice([0, 32, 64, 128, 100]) if c["out"] == "e4m3" else 0
        return c
    token = rng.random() < 0.3 and not op.endswith("bwd")
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    width = _log(rng, 32, 2048)
    if rng.random() < 0.6:
        width = max(32, width // 64 * 64)
    if token:
        B, L, ragged, slots = _log(rng, 1, 256), 1, 0, 0
        if rng.random() < 0.7:
            slots = B + rng.randint(0, 64)
    else:
        ragged = rng.choice([0, 0, rng.randint(1, 1000)])
        most = 4096 * 2048 * (1 if ragged or op == "scan_bwd" else 4) // width
        B = _log(rng, 1, 16)
        L = min(16384 if ragged else 8192, _log(rng, 2, max(3, most if ragged else most // B)))
        slots = B + rng.randint(0, 4) if not op.endswith("bwd") and rng.random() < 0.5 else 0
    if op.startswith("conv"):
        head = rng.choice([0, 0, 32]) if width % 32 == 0 else 0
        return dict(op=op, B=B, L=L, C=width, W=rng.choice([2, 3, 4, 4, 5, 8]), dtype=dtype, act=rng.random() < 0.8,
                    head_dim=head, slots=slots, ragged=ragged)
    return dict(op=op, B=B, L=L, D=width, N=rng.choice([8, 13, 16, 16, 16]), G=2 if width % 2 == 0 and rng.random() < 0.3 else 1, dtype=dtype,
                gate=rng.random() < 0.7, slots=slots, ragged=ragged)


def _lens(case):
    """Lengths of a packed batch: B numbers, an empty one among them where B > 2, that leave some rows behind them."""
    B, T = case["B"], case["L"]
    used = T - T // 50 if T > 50 else T
    weight = [1 + (case["ragged"] * 7919 + 131 * i * i) % 17 for i in range(B)]
    if B > 2:
        weight[B // 2] = 0
    lens = [used * w // sum(weight) for w in weight]
    lens[0] += used - sum(lens)
    return lens


def _slots(case):
    """Which slot each sequence has: distinct; in a decoding batch of more than four the last entry is padding (-1)."""
    B, S = case["B"], case["slots"]
    step = next(k for k in range(max(1, S // 3), S + 1) if math.gcd(k, S) == 1) if S > 1 else 1
    at = [(i * step) % S for i in range(B)]
    if case["L"] == 1 and B > 4:
        at[-1] = -1
    return at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)

    def normal(*shape, dtype="fp32", scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dtype])

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = dict(case=case)
    if case["op"].startswith("norm"):
        rows, d, r = case["rows"], case["d"], case["r_dtype"]
        s["w"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(DT[case["dtype"]])
        if case["op"] == "norm":
            s["x"] = normal(rows, d, dtype=case["dtype"])
            s["res"] = normal(rows, d, dtype=r, scale=2.0) if case["residual"] else None
        else:
            s["h"] = normal(rows, d, dtype=r, scale=2.0)
            s["dy"] = normal(rows, d, dtype=case["dtype"], scale=0.1)
            s["dres"] = normal(rows, d, dtype=r, scale=0.1) if case["residual"] else None
        return s
    B, L, dt = case["B"], case["L"], case["dtype"]
    lead = (L,) if case["ragged"] else (B, L)
    n = case["slots"] or B
    if case["ragged"]:
        ends = [0]
        for k in _lens(case):
            ends.append(ends[-1] + k)
        s["start"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["slots"]:
        s["slot"] = torch.tensor(_slots(case), dtype=torch.int32, device="cuda")
    if case["op"].startswith("conv"):
        C, W = case["C"], case["W"]
        s["x"] = normal(*lead, C, dtype=dt)
        s["w"] = uniform(-1, 1, C, W).mul(W ** -0.5).to(DT[dt])
        s["b"] = normal(C, dtype=dt, scale=0.1)
        s["state"] = normal(n, W - 1, C, dtype=dt)
        if case["op"] == "conv_bwd":
            s["dy"] = normal(*_y_shape(case), dtype=dt)
            s["dstate"] = normal(B, W - 1, C, scale=0.5)
        return s
    D, N, G = case["D"], case["N"], case["G"]
    s["x"] = normal(*lead, D, dtype=dt)
    s["dt"] = normal(*lead, D, dtype=dt, scale=0.5)
    step = torch.exp(uniform(math.log(1e-3), math.log(0.1), D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * normal(D, N))).contiguous()
    s["Bm"] = normal(*lead, G, N, dtype=dt)
    s["Cm"] = normal(*lead, G, N, dtype=dt)
    s["Dskip"] = 1 + 0.1 * normal(D)
    s["z"] = normal(*lead, D, dtype=dt) if case["gate"] else None
    s["h"] = normal(n, D, N, scale=0.2)
    if case["op"] == "scan_bwd":
        s["dy"] = normal(*lead, D, dtype=dt)
        s["dh"] = normal(B, D, N, scale=0.5)
    return s


def _y_shape(case):
    B, L, C, hd = case["B"], case["L"], case["C"], case["head_dim"]
    if not hd:
        return (L, C) if case["ragged"] else (B, L, C)
    return (C // hd, L, hd) if case["ragged"] else (B, C // hd, L, hd)


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "conv": _conv, "conv_bwd": _conv_bwd, "scan": _scan, "scan_bwd": _scan_bwd}[op](state)


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import test_memorization_recurrent_gb300 as A
    c, f = s["case"], _OWN[s["case"]["op"]]
    if "plan" not in s:  # the description, the outputs and the workspace, which a program keeps from step to step
        s["plan"] = f(A, s, c)
    return s["plan"]()


def _codes(A):
    return {"bf16": A.BF16, "fp16": A.F16, "fp32": A.F32, "e4m3": A.E4M3}


def _with_workspace(cfg, nbytes):
    ws = torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")
    cfg.workspace, cfg.workspace_bytes = ws.data_ptr(), nbytes
    return ws


def _own_norm(A, s, c):
    k = _codes(A)
    x, res = s["x"], s["res"]
    y = torch.empty(x.shape, device="cuda", dtype=torch.float8_e4m3fn if c["out"] == "e4m3" else DT[c["out"]])
    groups = -(-c["d"] // c["group"]) if c["group"] else 1
    scale = torch.empty(c["rows"], groups, device="cuda") if c["out"] == "e4m3" else None
    h = torch.empty_like(res) if c["residual"] else None
    cfg = A.make_norm_cfg(c["rows"], c["d"], dtype=k[c["dtype"]], r_dtype=k[c["r_dtype"]], w_dtype=k[c["dtype"]],
                          out_dtype=k[c["out"]], group=c["group"])
    out = {n: t for n, t in (("y", y), ("scale", scale), ("h", h)) if t is not None}

    def call():
        A.atlas_norm_forward(x, res, s["w"], cfg, y, h, scale)
        return out
    return call


def _own_norm_bwd(A, s, c):
    k = _codes(A)
    cfg = A.make_norm_cfg(c["rows"], c["d"], dtype=k[c["dtype"]], r_dtype=k[c["r_dtype"]], w_dtype=k[c["dtype"]])
    ws = _with_workspace(cfg, A.atlas_norm_backward_workspace_bytes(cfg))
    dx, dw = torch.empty_like(s["h"]), torch.empty(c["d"], device="cuda")

    def call(keep=ws):
        A.atlas_norm_backward(s["h"], s["w"], s["dy"], s["dres"], cfg, dx, dw)
        return {"dx": dx, "dw": dw}
    return call


def _conv_cfg(A, s, c):
    k = _codes(A)[c["dtype"]]
    return A.make_conv_cfg(c["B"], c["L"], c["C"], c["W"], act=A.ACT_SILU if c["act"] else A.ACT_NONE, dtype=k, w_dtype=k,
                           head_dim=c["head_dim"], seq_start=s.get("start"), slot=s.get("slot"), n_slots=c["slots"])


def _own_conv(A, s, c):
    cfg = _conv_cfg(A, s, c)
    y, new = torch.zeros(_y_shape(c), dtype=DT[c["dtype"]], device="cuda"), s["state"].clone()

    def call():
        A.atlas_conv_forward(s["x"], s["w"], s["b"], cfg, y, s["state"], new)
        return {"y": y, "state": new}
    return call


def _own_conv_bwd(A, s, c):
    cfg = _conv_cfg(A, s, c)
    ws = _with_workspace(cfg, A.atlas_conv_backward_workspace_bytes(cfg))
    dx = torch.zeros_like(s["x"])
    dw, db = torch.empty(c["C"], c["W"], device="cuda"), torch.empty(c["C"], device="cuda")

    def call(keep=ws):
        dstate = s["dstate"].clone()
        A.atlas_conv_backward(s["x"], s["w"], s["b"], cfg, s["state"], s["dy"], dstate, dx, dw, db)
        return {"dx": dx, "dw": dw, "db": db, "dstate": dstate}
    return call


def _scan_cfg(A, s, c):
    return A.make_scan_cfg(c["B"], c["L"], c["D"], c["N"], G=c["G"], dtype=_codes(A)[c["dtype"]], softplus=True,
                           seq_start=s.get("start"), slot=s.get("slot"), n_slots=c["slots"])


def _own_scan(A, s, c):
    cfg = _scan_cfg(A, s, c)
    ws = _with_workspace(cfg, A.atlas_scan_workspace_bytes(cfg))
    y, h = torch.zeros_like(s["x"]), s["h"].clone()

    def call(keep=ws):
        A.atlas_scan_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["z"], s["dt_bias"], cfg, y, s["h"], h)
        return {"y": y, "h": h}
    return call


def _own_scan_bwd(A, s, c):
    cfg = _scan_cfg(A, s, c)
    ws = _with_workspace(cfg, A.atlas_scan_backward_workspace_bytes(cfg))
    like = {"dx": "x", "ddt": "dt", "dB": "Bm", "dC": "Cm", "dz": "z", "dA": "A", "dD": "Dskip", "ddt_bias": "dt_bias"}
    o = {k: torch.zeros_like(s[v]) for k, v in like.items() if s[v] is not None}

    def call(keep=ws):
        dh = s["dh"].clone()
        A.atlas_scan_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["Dskip"], s["z"], s["dt_bias"], cfg, s["h"], s["dy"],
                              dh, o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], o["dD"], o.get("dz"), o["ddt_bias"])
        return dict(o, dh=dh)
    return call


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "conv": _own_conv, "conv_bwd": _own_conv_bwd, "scan": _own_scan,
        "scan_bwd": _own_scan_bwd}


# ---------------------------------------------------------------- the plain forms

EPS = 1e-6


def _norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
    out = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    if c["out"] != "e4m3":
        return dict(out, y=y.to(DT[c["out"]]))
    g = c["group"] or c["d"]
    y = torch.nn.functional.pad(y, (0, -c["d"] % g)).unflatten(-1, (-1, g))
    scale = y.abs().amax(-1).clamp_min(1e-30) * (1 / E4M3_MAX)
    q = (y * (1 / scale)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)[:, :c["d"]]
    return dict(out, y=q.to(torch.float8_e4m3fn), scale=scale)


def _norm_bwd(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["w"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    hat, wdy = h * r, dy * w
    dx = r * (wdy - hat * (wdy * hat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * hat).sum(0)}


def _rows(s):
    """Packed rows as [B, longest]: which row each place takes (its sequence's first where there is none) and which places hold one."""
    start = s["start"].long()
    n = start[1:] - start[:-1]
    at = torch.arange(max(1, max(_lens(s["case"]))), device="cuda")
    here = at < n[:, None]
    return (start[:-1, None] + at).where(here, torch.zeros_like(at)), here


def _padded(s, x):
    if "start" not in s:
        return x
    at, here = _rows(s)
    return x[at] * here.reshape(*here.shape, *[1] * (x.dim() - 1))


def _packed(s, y, like):
    """Back into rows; the rows behind the last sequence are zero."""
    if "start" not in s:
        return y.to(like.dtype)
    at, here = _rows(s)
    out = torch.zeros(like.shape, dtype=like.dtype, device="cuda")
    out[at[here]] = y[here].to(like.dtype)
    return out


def _length(s, x):
    """Tokens of each sequence, [B]."""
    c = s["case"]
    return s["start"].diff().long() if "start" in s else torch.full((c["B"],), c["L"], device="cuda")


def _taken(s, state):
    return state if "slot" not in s else state[s["slot"].long().clamp_min(0)]


def _given(s, state, new):
    if "slot" not in s:
        return new.to(state.dtype)
    at = s["slot"].long()
    out = state.clone()
    out[at[at >= 0]] = new[at >= 0].to(state.dtype)
    return out


def _skipped(s, y):
    """Zero where a decoding batch has padding."""
    return y if "slot" not in s else y * (s["slot"] >= 0).reshape(-1, *[1] * (y.dim() - 1))


def _heads(case, y):
    """[.., L, C] as the layout of y: head-major where the case has heads."""
    return y.unflatten(-1, (-1, case["head_dim"])).transpose(-2, -3) if case["head_dim"] else y


def _tail(s, x, rows):
    """The last `rows` of each sequence of x [B, rows + L, C] that has its initial rows in front."""
    at = _length(s, x)[:, None] + torch.arange(rows, device="cuda")
    return torch.gather(x, 1, at[..., None].expand(-1, -1, x.shape[-1]))


def _conv(s):
    c, W = s["case"], s["case"]["W"]
    x = torch.cat([_taken(s, s["state"]).float(), _padded(s, s["x"]).float()], 1)
    y = (x.unfold(1, W, 1) * s["w"].float()).sum(-1) + s["b"].float()
    if c["act"]:
        y = y * torch.sigmoid(y)
    y = _packed(s, _skipped(s, y), s["x"])
    return {"y": _heads(c, y).contiguous(), "state": _given(s, s["state"], _tail(s, x, W - 1))}


def _conv_bwd(s):
    c, W = s["case"], s["case"]["W"]
    dy = s["dy"].transpose(-2, -3).flatten(-2) if c["head_dim"] else s["dy"]
    dy = _padded(s, dy).float()
    x = torch.cat([s["state"].float(), _padded(s, s["x"]).float()], 1)
    w, windows = s["w"].float(), x.unfold(1, W, 1)
    if c["act"]:
        p = (windows * w).sum(-1) + s["b"].float()
        sig = torch.sigmoid(p)
        dy = dy * sig * (1 + p * (1 - sig))
    dw = (windows * dy[..., None]).sum((0, 1))
    dx = (torch.nn.functional.pad(dy, (0, 0, W - 1, W - 1)).unfold(1, W, 1) * w.flip(-1)).sum(-1)
    at = _length(s, x)[:, None] + torch.arange(W - 1, device="cuda")
    dx = dx.scatter_add(1, at[..., None].expand(-1, -1, x.shape[-1]), s["dstate"])
    return {"dx": _packed(s, dx[:, W - 1:], s["x"]), "dw": dw, "db": dy.sum((0, 1)), "dstate": dx[:, :W - 1].contiguous()}


def _prefix(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1 by doubling: after a step every place holds the sum over twice as many tokens."""
    shift, L = 1, a.shape[1]
    while shift < L:
        u = torch.cat([u[:, :shift], torch.addcmul(u[:, shift:], a[:, shift:], u[:, :-shift])], 1)
        a = torch.cat([a[:, :shift], a[:, shift:] * a[:, :-shift]], 1)
        shift *= 2
    return u


def _scan_terms(s):
    """What both directions begin with, [B, L, ..] in 32 bits: x, dt, softplus' slope, decays, dt B x, B and C for every channel's group, the state in front."""
    c = s["case"]
    x, Bm, Cm = (_padded(s, s[k]).float() for k in ("x", "Bm", "Cm"))
    raw = s["dt"].float() + s["dt_bias"]
    dt = _padded(s, torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp_max(20)))))  # zero behind a sequence: the state stays
    each = c["D"] // c["G"]
    Bm, Cm = (m.repeat_interleave(each, -2) for m in (Bm, Cm)) if c["G"] > 1 else (Bm, Cm)
    a = torch.exp(dt[..., None] * s["A"])
    u = (dt * x)[..., None] * Bm
    h0 = _taken(s, s["h"])
    u[:, 0] += a[:, 0] * h0
    return x, dt, _padded(s, torch.sigmoid(raw)), a, u, Bm, Cm, h0


def _scan(s):
    x, dt, _, a, u, Bm, Cm, h0 = _scan_terms(s)
    h = _prefix(a, u)
    y = (h * Cm).sum(-1) + s["Dskip"] * x
    if s["z"] is not None:
        z = _padded(s, s["z"]).float()
        y = y * z * torch.sigmoid(z)
    return {"y": _packed(s, _skipped(s, y), s["x"]), "h": _given(s, s["h"], h[:, -1])}


def _scan_bwd(s):
    c = s["case"]
    x, dt, slope, a, u, Bm, Cm, h0 = _scan_terms(s)
    B, L, D, N, G = *x.shape, c["N"], c["G"]
    h = _prefix(a, u)
    dy, out = _padded(s, s["dy"]).float(), {}
    if s["z"] is not None:
        z = _padded(s, s["z"]).float()
        sig = torch.sigmoid(z)
        y = (h * Cm).sum(-1) + s["Dskip"] * x
        out["dz"] = _packed(s, dy * y * sig * (1 + z * (1 - sig)), s["z"])
        dy = dy * z * sig
    # g_t = C_t dy_t + a_{t+1} g_{t+1}, the same recurrence backwards
    v = dy[..., None] * Cm
    v[:, -1] += s["dh"]
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _prefix(later.flip(1), v.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    q = g * a * before
    gB = (g * Bm).sum(-1)
    ddt = (q * s["A"]).sum(-1) + gB * x
    draw = ddt * slope
    out["dx"] = _packed(s, gB * dt + s["Dskip"] * dy, s["x"])
    out["ddt"] = _packed(s, draw, s["dt"])
    out["dB"] = _packed(s, (g * (dt * x)[..., None]).unflatten(2, (G, -1)).sum(3), s["Bm"])
    out["dC"] = _packed(s, (h * dy[..., None]).unflatten(2, (G, -1)).sum(3), s["Cm"])
    out["dA"] = (q * dt[..., None]).sum((0, 1))
    out["dD"] = (dy * x).sum((0, 1))
    out["ddt_bias"] = draw.sum((0, 1))
    out["dh"] = a[:, 0] * g[:, 0]
    return out


# ---------------------------------------------------------------- what is to be read, written and computed

def work(case):
    c = case
    if c["op"].startswith("norm"):
        n, e, r = c["rows"] * c["d"], SIZE[c["dtype"]], SIZE[c["r_dtype"]]
        if c["op"] == "norm":
            groups = -(-c["d"] // c["group"]) if c["group"] else 1
            q = c["rows"] * groups * 4 if c["out"] == "e4m3" else 0
            return {"bytes": n * (e + SIZE[c["out"]] + (2 * r if c["residual"] else 0)) + q + c["d"] * e, "flops": 6 * n}
        return {"bytes": n * (2 * r + e + (r if c["residual"] else 0)) + c["d"] * (e + 4), "flops": 12 * n}
    e, B = SIZE[c["dtype"]], c["B"]
    tokens = sum(_lens(c)) if c["ragged"] else B * c["L"]
    if c["op"].startswith("conv"):
        C, W = c["C"], c["W"]
        n, state = tokens * C, B * (W - 1) * C
        if c["op"] == "conv":
            return {"bytes": (2 * n + 2 * state + C * (W + 1)) * e, "flops": n * (2 * W + 5)}
        return {"bytes": (3 * n + state + C * (W + 1)) * e + (2 * state + C * (W + 1)) * 4, "flops": n * (6 * W + 9)}
    D, N, G = c["D"], c["N"], c["G"]
    n, bc, state = tokens * D, 2 * tokens * G * N, B * D * N * 4
    z = 1 if c["gate"] else 0
    if c["op"] == "scan":
        return {"bytes": (n * (3 + z) + bc) * e + 2 * state + D * (N + 2) * 4, "flops": n * (8 * N + 12)}
    return {"bytes": (n * (5 + 2 * z) + 2 * bc) * e + 3 * state + 2 * D * (N + 2) * 4, "flops": n * (24 * N + 30)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions, token by token and tap by tap in 64 bits; outputs are not rounded to their types."""
    s, c = prepare(case, seed), case
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if c["op"].startswith("norm"):
        return _exact_norm(d, c)
    if c["ragged"]:
        lens = _lens(c)
        first = [sum(lens[:b]) for b in range(c["B"])]
    else:
        lens, first = [c["L"]] * c["B"], None
    slot = _slots(c) if c["slots"] else list(range(c["B"]))
    return (_exact_conv if c["op"].startswith("conv") else _exact_scan)(d, c, lens, first, slot)


def _exact_norm(d, c):
    h = d["h"] if "h" in d else d["x"] if d["res"] is None else d["x"] + d["res"]
    rms = torch.linalg.vector_norm(h, dim=1, keepdim=True).square().div(c["d"]).add(EPS).sqrt()
    if c["op"] == "norm":
        y = h / rms * d["w"]
        out = {} if d["res"] is None else {"h": h}
        if c["out"] != "e4m3":
            return dict(out, y=y)
        g = c["group"] or c["d"]
        scale = torch.stack([p.abs().max(1).values.clamp_min(1e-30) / E4M3_MAX for p in y.split(g, 1)], 1)
        return dict(out, y=torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(y.split(g, 1))], 1), scale=scale)
    v = d["dy"] * d["w"]
    dx = v / rms - h * ((v * h).sum(1, keepdim=True) / (c["d"] * rms ** 3))
    if d["dres"] is not None:
        dx += d["dres"]
    return {"dx": dx, "dw": torch.einsum("rc,rc->c", d["dy"], h / rms)}


def _exact_conv(d, c, lens, first, slot):
    W, C, bwd = c["W"], c["C"], c["op"] == "conv_bwd"
    flat = lambda t: t.movedim(-3, -2).flatten(-2) if c["head_dim"] else t  # noqa: E731
    y, state = torch.zeros_like(d["x"]), d["state"].clone()
    dx, dstate = torch.zeros_like(d["x"]), torch.zeros(c["B"], W - 1, C, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros(C, W, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = slice(first[b], first[b] + n) if first else (b, slice(0, n))
        if slot[b] < 0:
            continue
        x = torch.cat([d["state"][slot[b]], d["x"][at]])
        p = d["b"] + sum(x[k:k + n] * d["w"][:, k] for k in range(W))
        y[at] = p / (1 + torch.exp(-p)) if c["act"] else p
        state[slot[b]] = x[n:]
        if bwd:
            g = flat(d["dy"])[at]
            if c["act"]:
                e = torch.exp(-p)
                g = g * (1 / (1 + e) + p * e / (1 + e) ** 2)
            full = torch.zeros_like(x)
            full[n:] += d["dstate"][b]
            for k in range(W):
                full[k:k + n] += g * d["w"][:, k]
                dw[:, k] += (g * x[k:k + n]).sum(0)
            db += g.sum(0)
            dstate[b], dx[at] = full[:W - 1], full[W - 1:]
    if bwd:
        return {"dx": dx, "dw": dw, "db": db, "dstate": dstate}
    return {"y": _heads(c, y), "state": state}


def _exact_scan(d, c, lens, first, slot):
    D, N, G, bwd, f64 = c["D"], c["N"], c["G"], c["op"] == "scan_bwd", dict(dtype=torch.float64, device="cuda")
    raw = d["dt"] + d["dt_bias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    z, lead = d["z"], d["x"].shape[:-1]
    gate = z / (1 + torch.exp(-z)) if z is not None else torch.ones_like(d["x"])
    at = [torch.arange(n, device="cuda") + first[b] if first else torch.arange(n, device="cuda") + b * c["L"] for b, n in enumerate(lens)]
    flat = lambda t: t.reshape(-1, *t.shape[len(lead):])  # noqa: E731
    xs, ds, Bs, Cs, gs = (flat(t) for t in (d["x"], dt, d["Bm"], d["Cm"], gate))
    core, h_end = torch.zeros_like(xs), d["h"].clone()  # core: C h + D x, before the gate
    live = [b for b in range(c["B"]) if slot[b] >= 0]
    if not bwd and c["slots"] == 0 and not first:  # sequences of one length go together
        h = d["h"].clone()
        x3, d3, B3, C3 = (t.unflatten(0, (c["B"], c["L"])) for t in (xs, ds, Bs, Cs))
        y3 = torch.empty_like(x3)
        for t in range(c["L"]):
            h = torch.exp(d3[:, t, :, None] * d["A"]) * h
            h = h.unflatten(1, (G, -1)).addcmul_((d3[:, t] * x3[:, t]).unflatten(1, (G, -1))[..., None], B3[:, t, :, None, :]).flatten(1, 2)
            y3[:, t] = torch.matmul(h.unflatten(1, (G, -1)), C3[:, t, :, :, None]).flatten(1)
        y = (y3.flatten(0, 1) + d["Dskip"] * xs) * gs
        return {"y": y.reshape(d["x"].shape), "h": h}
    o = {k: torch.zeros_like(flat(d[v])) for k, v in (("dx", "x"), ("ddt", "dt"), ("dB", "Bm"), ("dC", "Cm"))} if bwd else {}
    dA, dh = torch.zeros(D, N, **f64), torch.zeros(c["B"], D, N, **f64)
    grouped = lambda v: v.unflatten(0, (G, -1))  # noqa: E731
    if bwd:
        dys = flat(d["dy"]) * gs
    for b in live:
        h, steps = d["h"][slot[b]], at[b].tolist()
        path = torch.empty(len(steps) + 1, D, N, **f64) if bwd else None
        if bwd:
            path[0] = h
        for i, t in enumerate(steps):
            h = torch.exp(ds[t][:, None] * d["A"]) * h + (grouped(ds[t] * xs[t])[..., None] * Bs[t][:, None, :]).flatten(0, 1)
            core[t] = (grouped(h) * Cs[t][:, None, :]).sum(-1).flatten()
            if bwd:
                path[i + 1] = h
        h_end[slot[b]] = h
        if not bwd:
            continue
        g = d["dh"][b]
        for i in reversed(range(len(steps))):
            t = steps[i]
            g = g + (grouped(dys[t])[..., None] * Cs[t][:, None, :]).flatten(0, 1)
            o["dC"][t] = (grouped(path[i + 1]) * grouped(dys[t])[..., None]).sum(1)
            o["dB"][t] = (grouped(g) * grouped(ds[t] * xs[t])[..., None]).sum(1)
            gB = (grouped(g) * Bs[t][:, None, :]).sum(-1).flatten()
            g = g * torch.exp(ds[t][:, None] * d["A"])
            q = g * path[i]
            o["ddt"][t] = gB * xs[t] + (q * d["A"]).sum(-1)
            o["dx"][t] = gB * ds[t]
            dA += q * ds[t][:, None]
        dh[b] = g
    core += d["Dskip"] * xs
    if not bwd:
        skip = torch.zeros(xs.shape[0], 1, **f64)
        for b in live:
            skip[at[b]] = 1
        return {"y": (core * gs * skip).reshape(d["x"].shape), "h": h_end}
    used = torch.zeros(xs.shape[0], 1, **f64)
    for b in live:
        used[at[b]] = 1
    draw = o["ddt"] / (1 + torch.exp(-flat(raw))) * used
    out = {"dx": (o["dx"] + d["Dskip"] * dys * used).reshape(d["x"].shape), "ddt": draw.reshape(d["x"].shape),
           "dB": o["dB"].reshape(d["Bm"].shape), "dC": o["dC"].reshape(d["Cm"].shape), "dA": dA,
           "dD": (dys * xs * used).sum(0), "ddt_bias": draw.sum(0), "dh": dh}
    if z is not None:
        e = torch.exp(-flat(z))
        out["dz"] = (flat(d["dy"]) * core * used * (1 / (1 + e) + flat(z) * e / (1 + e) ** 2)).reshape(d["x"].shape)
    return out
