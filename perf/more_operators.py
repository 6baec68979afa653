"""Layer norm and a gated linear recurrence, as cases to time and compare.

layernorm  residual addition, mean and variance of a row, weight and bias; the output in bf16 / fp16 / fp32
           or e4m3 with one scale per row or per group of channels; its backward pass with dw and db
glr        gated linear recurrence, one state a channel:
               s_t = c softplus(lambda) sigmoid(r_t + rb),  a_t = exp(-s_t)
               h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + ib) x_t,  y_t = h_t SiLU(z_t)
           for prompts, packed prompts and single tokens, its state carried; its training pass (forward,
           then backward)

`run` computes them in plain torch operations, or (own = True) through this repository's entry points.
The largest cases have the tokens and the width of the DeltaNet-like workload (8 sequences x 4096 tokens,
16 heads x 128).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-5
SHARP = 8.0  # c


def listed():
    return [
        # the tokens of one decoding step entering a layer
        dict(name="ln-token", op="ln", rows=8, d=2048, dtype="bf16", r_dtype="bf16", out="bf16", group=0, residual=True),
        # every token of the prompts entering a layer whose projections take 8 bits, scales per 128 channels
        dict(name="ln-prompt", op="ln", rows=32768, d=2048, dtype="bf16", r_dtype="bf16", out="e4m3", group=128, residual=True),
        # the memory's readouts (32 bits) of all heads and tokens, each normalised over its 128 channels
        dict(name="ln-heads", op="ln", rows=524288, d=128, dtype="fp32", r_dtype="fp32", out="bf16", group=0, residual=False),
        # rows of odd width, none but the first of which starts on a boundary of 16 bytes
        dict(name="ln-odd", op="ln", rows=20000, d=1371, dtype="fp16", r_dtype="fp16", out="fp16", group=0, residual=True),
        # the training pass with a residual stream held in 32 bits
        dict(name="ln-train", op="ln_bwd", rows=16384, d=2560, dtype="bf16", r_dtype="fp32", residual=True),
        # the training pass at an odd width
        dict(name="ln-train-odd", op="ln_bwd", rows=12001, d=1371, dtype="bf16", r_dtype="bf16", residual=False),
        # one decoding step of 64 sequences whose states lie in a larger pool
        dict(name="glr-token", op="glr", B=64, L=1, D=2048, dtype="bf16", gate=True, slots=96, ragged=0),
        # prompts
        dict(name="glr-prompt", op="glr", B=8, L=4096, D=2048, dtype="bf16", gate=True, slots=0, ragged=0),
        # one long document: little parallel work but the length
        dict(name="glr-long", op="glr", B=1, L=65536, D=512, dtype="bf16", gate=False, slots=0, ragged=0),
        # a packed batch of prompts of unequal lengths, odd width, with states carried on
        dict(name="glr-packed", op="glr", B=11, L=9001, D=1500, dtype="fp16", gate=True, slots=16, ragged=5),
        # the training pass
        dict(name="glr-train", op="glr_train", B=8, L=4096, D=2048, dtype="bf16", gate=True, slots=0, ragged=0),
        # the training pass of packed documents in 32 bits, odd width
        dict(name="glr-train-packed", op="glr_train", B=7, L=8192, D=1111, dtype="fp32", gate=True, slots=0, ragged=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_bwd", "glr", "glr", "glr_train"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op.startswith("ln"):
        d = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            d = max(8, d // 16 * 16)
        rows = _log(rng, 1, max(2, min(524288, 32768 * 2048 // d)))
        c = dict(op=op, rows=rows, d=d, dtype=dtype)
        c["residual"] = rng.random() < 0.7
        c["r_dtype"] = rng.choice([dtype, "fp32"]) if c["residual"] else dtype
        if op == "ln":
            c["out"] = rng.choice([dtype, dtype, "bf16", "e4m3"])
            c["group"] = rng.choice([0, 32, 64, 128, 100]) if c["out"] == "e4m3" else 0
        return c
    D = _log(rng, 16, 4096)
    if rng.random() < 0.6:
        D = max(16, D // 16 * 16)
    gate = rng.random() < 0.7
    if op == "glr" and rng.random() < 0.3:
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, L=1, D=D, dtype=dtype, gate=gate, slots=B + rng.randint(0, 64) if rng.random() < 0.7 else 0, ragged=0)
    ragged = rng.choice([0, 0, rng.randint(1, 1000)])
    B = _log(rng, 1, 16)
    most = 8 * 4096 * 2048 // (D * (1 if ragged else B) * (2 if dtype == "fp32" else 1))
    L = _log(rng, 2, max(3, min(65536, most)))
    slots = B + rng.randint(0, 4) if op == "glr" and rng.random() < 0.5 else 0
    return dict(op=op, B=B, L=L, D=D, dtype=dtype, gate=gate, slots=slots, ragged=ragged)


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
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape, dtype="fp32", scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dtype])

    s = dict(case=case)
    if case["op"].startswith("ln"):
        rows, d, dt, r = case["rows"], case["d"], case["dtype"], case["r_dtype"]
        s["w"] = (1 + 0.1 * normal(d)).to(DT[dt])
        s["b"] = normal(d, dtype=dt, scale=0.1)
        mean = 0.5 * normal(rows, 1)  # rows whose mean is not zero
        if case["op"] == "ln":
            s["x"] = (normal(rows, d) + mean).to(DT[dt])
            s["res"] = normal(rows, d, dtype=r, scale=2.0) if case["residual"] else None
        else:
            s["h"] = (normal(rows, d, scale=2.0) + mean).to(DT[r])
            s["dy"] = normal(rows, d, dtype=dt, scale=0.1)
            s["dres"] = normal(rows, d, dtype=r, scale=0.1) if case["residual"] else None
        return s
    B, L, D, dt = case["B"], case["L"], case["D"], case["dtype"]
    lead = (L,) if case["ragged"] else (B, L)
    if case["ragged"]:
        ends = [0]
        for k in _lens(case):
            ends.append(ends[-1] + k)
        s["start"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if case["slots"]:
        s["slot"] = torch.tensor(_slots(case), dtype=torch.int32, device="cuda")
    for k in ("x", "r", "i"):
        s[k] = normal(*lead, D, dtype=dt)
    s["z"] = normal(*lead, D, dtype=dt) if case["gate"] else None
    slowest = torch.rand(D, generator=g, device="cuda") * 0.099 + 0.9  # exp(-c softplus(lambda)): decays from 0.9 to 0.999
    s["lam"] = torch.log(torch.expm1(-torch.log(slowest) / SHARP))
    s["rb"], s["ib"] = normal(D, scale=0.1), normal(D, scale=0.1)
    s["h"] = normal(case["slots"] or B, D, scale=0.5)
    if case["op"] == "glr_train":
        s["dy"] = normal(*lead, D, dtype=dt)
        s["dh"] = normal(B, D, scale=0.5)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return {"ln": _ln, "ln_bwd": _ln_bwd, "glr": _glr, "glr_train": _glr_train}[op](state)


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import test_memorization_recurrent_gb300 as A
    c = s["case"]
    if "plan" not in s:  # the description, the outputs and the workspace, which a program keeps from step to step
        s["plan"] = {"ln": _own_ln, "ln_bwd": _own_ln_bwd, "glr": _own_glr, "glr_train": _own_glr_train}[c["op"]](A, s, c)
    return s["plan"]()


def _codes(A):
    return {"bf16": A.BF16, "fp16": A.F16, "fp32": A.F32, "e4m3": A.E4M3}


def _space(nbytes):
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device="cuda")


def _with_workspace(cfg, nbytes):
    ws = _space(nbytes)
    cfg.workspace, cfg.workspace_bytes = ws.data_ptr(), nbytes
    return ws


def _own_ln(A, s, c):
    k = _codes(A)
    x, res = s["x"], s["res"]
    y = torch.empty(x.shape, device="cuda", dtype=torch.float8_e4m3fn if c["out"] == "e4m3" else DT[c["out"]])
    groups = -(-c["d"] // c["group"]) if c["group"] else 1
    scale = torch.empty(c["rows"], groups, device="cuda") if c["out"] == "e4m3" else None
    h = torch.empty_like(res) if c["residual"] else None
    cfg = A.make_norm_cfg(c["rows"], c["d"], dtype=k[c["dtype"]], r_dtype=k[c["r_dtype"]], w_dtype=k[c["dtype"]],
                          out_dtype=k[c["out"]], group=c["group"], eps=EPS)
    out = {n: t for n, t in (("y", y), ("scale", scale), ("h", h)) if t is not None}

    def call():
        A.atlas_layernorm_forward(x, res, s["w"], s["b"], cfg, y, h, scale)
        return out
    return call


def _own_ln_bwd(A, s, c):
    k = _codes(A)
    cfg = A.make_norm_cfg(c["rows"], c["d"], dtype=k[c["dtype"]], r_dtype=k[c["r_dtype"]], w_dtype=k[c["dtype"]], eps=EPS)
    ws = _with_workspace(cfg, A.atlas_layernorm_backward_workspace_bytes(cfg))
    dx, dw, db = torch.empty_like(s["h"]), torch.empty(c["d"], device="cuda"), torch.empty(c["d"], device="cuda")

    def call(keep=ws):
        A.atlas_layernorm_backward(s["h"], s["w"], s["dy"], s["dres"], cfg, dx, dw, db)
        return {"dx": dx, "dw": dw, "db": db}
    return call


def _glr_cfg(A, s, c):
    return A.make_glr_cfg(c["B"], c["L"], c["D"], c=SHARP, dtype=_codes(A)[c["dtype"]], seq_start=s.get("start"),
                          slot=s.get("slot"), n_slots=c["slots"])


def _own_glr(A, s, c):
    cfg = _glr_cfg(A, s, c)
    ws = _with_workspace(cfg, A.atlas_glr_workspace_bytes(cfg))
    y, h = torch.zeros_like(s["x"]), s["h"].clone()

    def call(keep=ws):
        A.atlas_glr_forward(s["x"], s["r"], s["i"], s["z"], s["lam"], s["rb"], s["ib"], cfg, y, s["h"], h)
        return {"y": y, "h": h}
    return call


def _own_glr_train(A, s, c):
    cfg = _glr_cfg(A, s, c)
    ws = _with_workspace(cfg, max(A.atlas_glr_workspace_bytes(cfg), A.atlas_glr_backward_workspace_bytes(cfg)))
    kept = _space(A.atlas_glr_kept_bytes(cfg))  # what the forward pass leaves for the backward pass
    y, h = torch.zeros_like(s["x"]), torch.empty_like(s["h"])
    o = {k: torch.zeros_like(s[v]) for k, v in (("dx", "x"), ("dr", "r"), ("di", "i"), ("dz", "z")) if s[v] is not None}
    o.update((k, torch.empty(c["D"], device="cuda")) for k in ("dlam", "drb", "dib"))

    def call(keep=ws):
        dh = s["dh"].clone()
        A.atlas_glr_forward(s["x"], s["r"], s["i"], s["z"], s["lam"], s["rb"], s["ib"], cfg, y, s["h"], h, kept)
        A.atlas_glr_backward(s["x"], s["r"], s["i"], s["z"], s["lam"], s["rb"], s["ib"], cfg, s["h"], kept, s["dy"], dh,
                             o["dx"], o["dr"], o["di"], o.get("dz"), o["dlam"], o["drb"], o["dib"])
        return dict(o, y=y, h=h, dh=dh)
    return call


# ---------------------------------------------------------------- the plain forms

def _ln(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    mid = h - h.mean(-1, keepdim=True)
    y = mid * torch.rsqrt(mid.square().mean(-1, keepdim=True) + EPS) * s["w"].float() + s["b"].float()
    out = {} if s["res"] is None else {"h": h.to(s["res"].dtype)}
    if c["out"] != "e4m3":
        return dict(out, y=y.to(DT[c["out"]]))
    g = c["group"] or c["d"]
    y = torch.nn.functional.pad(y, (0, -c["d"] % g)).unflatten(-1, (-1, g))
    scale = y.abs().amax(-1).clamp_min(1e-30) * (1 / E4M3_MAX)
    q = (y * (1 / scale)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)[:, :c["d"]]
    return dict(out, y=q.to(torch.float8_e4m3fn), scale=scale)


def _ln_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    mid = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt(mid.square().mean(-1, keepdim=True) + EPS)
    hat, wdy = mid * r, dy * s["w"].float()
    dx = r * (wdy - wdy.mean(-1, keepdim=True) - hat * (wdy * hat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * hat).sum(0), "db": dy.sum(0)}


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
    return x[at] * here[..., None]


def _packed(s, y, like):
    """Back into rows; the rows behind the last sequence are zero."""
    if "start" not in s:
        return y.to(like.dtype)
    at, here = _rows(s)
    out = torch.zeros(like.shape, dtype=like.dtype, device="cuda")
    out[at[here]] = y[here].to(like.dtype)
    return out


def _taken(s, state):
    return state if "slot" not in s else state[s["slot"].long().clamp_min(0)]


def _given(s, state, new):
    if "slot" not in s:
        return new
    at = s["slot"].long()
    out = state.clone()
    out[at[at >= 0]] = new[at >= 0]
    return out


def _prefix(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1 by doubling: after a step every place holds the sum over twice as many tokens."""
    shift, L = 1, a.shape[1]
    while shift < L:
        u = torch.cat([u[:, :shift], torch.addcmul(u[:, shift:], a[:, shift:], u[:, :-shift])], 1)
        a = torch.cat([a[:, :shift], a[:, shift:] * a[:, :-shift]], 1)
        shift *= 2
    return u


def _softplus(x):
    return torch.clamp_min(x, 0) + torch.log1p(torch.exp(-x.abs()))


def _glr_terms(s):
    """What both directions begin with, [B, L, D] in 32 bits; behind a sequence's end s = 0 and nothing enters, so the state stays."""
    x = _padded(s, s["x"]).float()
    sr = torch.sigmoid(_padded(s, s["r"]).float() + s["rb"])
    si = torch.sigmoid(_padded(s, s["i"]).float() + s["ib"])
    step = SHARP * _softplus(s["lam"]) * sr
    if "start" in s:
        step = step * _rows(s)[1][..., None]
    a, beta = torch.exp(-step), torch.sqrt(-torch.expm1(-2 * step))
    u, h0 = beta * si * x, _taken(s, s["h"])
    lead = u.clone()
    lead[:, 0] += a[:, 0] * h0
    return x, sr, si, step, a, beta, h0, _prefix(a, lead)


def _glr(s):
    h = _glr_terms(s)[-1]
    y = h
    if s["z"] is not None:
        z = _padded(s, s["z"]).float()
        y = h * z * torch.sigmoid(z)
    if "slot" in s:
        y = y * (s["slot"] >= 0).reshape(-1, 1, 1)
    return {"y": _packed(s, y, s["x"]), "h": _given(s, s["h"], h[:, -1])}


def _glr_train(s):
    x, sr, si, step, a, beta, h0, h = _glr_terms(s)
    dy, out, y = _padded(s, s["dy"]).float(), {}, h
    if s["z"] is not None:
        z = _padded(s, s["z"]).float()
        sz = torch.sigmoid(z)
        y = h * z * sz
        out["dz"] = _packed(s, dy * h * sz * (1 + z * (1 - sz)), s["z"])
        dy = dy * z * sz
    out["y"], out["h"] = _packed(s, y, s["x"]), h[:, -1].clone()
    # g_t = dy_t + a_{t+1} g_{t+1}: the same recurrence backwards
    v = dy.clone()
    v[:, -1] += s["dh"]
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _prefix(later.flip(1), v.flip(1)).flip(1)
    before = torch.cat([h0[:, None], h[:, :-1]], 1)
    slope = g * step * (si * x * a * a / beta.clamp_min(1e-30) - a * before)  # s dL/ds
    dr, gb = slope * (1 - sr), g * beta * si
    di = gb * x * (1 - si)
    out["dx"], out["dr"], out["di"] = (_packed(s, t, s["x"]) for t in (gb, dr, di))
    out["dlam"] = slope.sum((0, 1)) * torch.sigmoid(s["lam"]) / _softplus(s["lam"])
    out["drb"], out["dib"] = dr.sum((0, 1)), di.sum((0, 1))
    out["dh"] = a[:, 0] * g[:, 0]
    return out


# ---------------------------------------------------------------- what is to be read, written and computed

def work(case):
    c = case
    if c["op"].startswith("ln"):
        n, e, r = c["rows"] * c["d"], SIZE[c["dtype"]], SIZE[c["r_dtype"]]
        if c["op"] == "ln":
            groups = -(-c["d"] // c["group"]) if c["group"] else 1
            q = c["rows"] * groups * 4 if c["out"] == "e4m3" else 0
            return {"bytes": n * (e + SIZE[c["out"]] + (2 * r if c["residual"] else 0)) + q + 2 * c["d"] * e, "flops": 9 * n}
        return {"bytes": n * (2 * r + e + (r if c["residual"] else 0)) + c["d"] * (e + 8), "flops": 17 * n}
    e, B, D = SIZE[c["dtype"]], c["B"], c["D"]
    n = (sum(_lens(c)) if c["ragged"] else B * c["L"]) * D
    z = 1 if c["gate"] else 0
    forward = n * (4 + z) * e + 2 * B * D * 4 + 3 * D * 4
    if c["op"] == "glr":
        return {"bytes": forward, "flops": n * 24}
    return {"bytes": forward + n * (7 + 2 * z) * e + 3 * B * D * 4 + 6 * D * 4, "flops": n * 80}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in 64 bits, the recurrence token by token; outputs are not rounded to their types."""
    s, c = prepare(case, seed), case
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return _exact_ln(d, c) if c["op"].startswith("ln") else _exact_glr(d, c)


def _exact_ln(d, c):
    h = d["h"] if "h" in d else d["x"] if d["res"] is None else d["x"] + d["res"]
    n = c["d"]
    mid = h - torch.einsum("rc->r", h)[:, None] / n
    std = torch.sqrt(torch.linalg.vector_norm(mid, dim=1, keepdim=True) ** 2 / n + EPS)
    if c["op"] == "ln":
        y = mid / std * d["w"] + d["b"]
        out = {} if d["res"] is None else {"h": h}
        if c["out"] != "e4m3":
            return dict(out, y=y)
        g = c["group"] or n
        scale = torch.stack([p.abs().max(1).values.clamp_min(1e-30) / E4M3_MAX for p in y.split(g, 1)], 1)
        return dict(out, y=torch.cat([p / scale[:, k:k + 1] for k, p in enumerate(y.split(g, 1))], 1), scale=scale)
    v = d["dy"] * d["w"]
    mean = torch.einsum("rc->r", v)[:, None] / n
    dx = (v - mean) / std - mid * (torch.einsum("rc,rc->r", v, mid)[:, None] / (n * std ** 3))
    if d["dres"] is not None:
        dx += d["dres"]
    return {"dx": dx, "dw": torch.einsum("rc,rc->c", d["dy"], mid / std), "db": torch.einsum("rc->c", d["dy"])}


def _exact_glr(d, c):
    B, D, train = c["B"], c["D"], c["op"] == "glr_train"
    lens = _lens(c) if c["ragged"] else [c["L"]] * B
    slot = _slots(c) if c["slots"] else list(range(B))
    new = {k: torch.zeros_like(d["x"]) for k in (("y", "dx", "dr", "di") if train else ("y",)) + (("dz",) if train and c["gate"] else ())}
    end, dh = d["h"].clone(), torch.zeros(B, D, dtype=torch.float64, device="cuda")
    sums = torch.zeros(3, D, dtype=torch.float64, device="cuda")
    rate = torch.logaddexp(d["lam"], torch.zeros_like(d["lam"]))
    if c["ragged"]:  # one sequence after the other, each [n, 1, D]
        first = [sum(lens[:b]) for b in range(B)]
        groups = [([b], slice(first[b], first[b] + lens[b])) for b in range(B)]
        take, put = (lambda t, at: t[at][:, None]), (lambda t, at, v: t.__setitem__(at, v[:, 0]))
    else:  # all together, [L, B, D], without padding
        live = [b for b in range(B) if slot[b] >= 0]
        groups = [(live, live)]
        take, put = (lambda t, at: t[at].transpose(0, 1)), (lambda t, at, v: t.__setitem__(at, v.transpose(0, 1)))
    for who, at in groups:
        own_slot = [slot[b] for b in who]
        h0 = h = d["h"][own_slot]
        x = take(d["x"], at)
        n = x.shape[0]
        er, ei = torch.exp(-(take(d["r"], at) + d["rb"])), torch.exp(-(take(d["i"], at) + d["ib"]))
        pull = SHARP * rate / (1 + er)
        a = torch.exp(-pull)
        beta = torch.sqrt(-torch.expm1(-2 * pull))
        u = beta * x / (1 + ei)
        path = torch.empty_like(u)
        for t in range(n):
            h = torch.addcmul(u[t], a[t], h, out=path[t])
        end[own_slot] = h
        gate = slope = None
        if c["gate"]:
            z = take(d["z"], at)
            ez = torch.exp(-z)
            gate, slope = z / (1 + ez), 1 / (1 + ez) + z * ez / (1 + ez) ** 2
        put(new["y"], at, path * gate if c["gate"] else path)
        if not train:
            continue
        v = take(d["dy"], at)
        if c["gate"]:
            put(new["dz"], at, v * path * slope)
            v = v * gate
        back, g = torch.empty_like(u), d["dh"][who]
        for t in reversed(range(n)):
            g = torch.add(v[t], g, out=back[t])
            g = a[t] * g
        dh[who] = g
        before = torch.cat([h0[None], path[:-1]]) if n else path
        da = back * before  # dL/da where u is held, and of u where it is not
        ds = -a * da + torch.where(beta > 0, back * x / (1 + ei) * a * a / beta, torch.zeros_like(beta))
        dr, di = ds * pull * er / (1 + er), back * u * ei / (1 + ei)
        put(new["dx"], at, back * beta / (1 + ei))
        put(new["dr"], at, dr)
        put(new["di"], at, di)
        sums += torch.stack([(ds * SHARP / (1 + er)).sum((0, 1)) / (1 + torch.exp(-d["lam"])), dr.sum((0, 1)), di.sum((0, 1))])
    if not train:
        return {"y": new["y"], "h": end}
    return dict(new, h=end, dh=dh, dlam=sums[0], drb=sums[1], dib=sums[2])
