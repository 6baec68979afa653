"""The gated linear recurrence on the GPU where blocks, warps and tiles meet.  References and tolerances as in
test_gpu_glr.py."""
import numpy as np
import pytest

import more_ops_ref as R

torch = pytest.importorskip("torch")
import test_memorization_recurrent_gb300 as A  # noqa: E402
from test_gpu_glr import C, Glr, check_grads, kept_of  # noqa: E402
from test_gpu_layer_ops import CODE, DT, TYPES, _lib, close, dev, draw, host, packed, rng, space, status  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,L,D", [(8, 640, 1024), (1, 6000, 512), (300, 3, 520)])
def test_every_warp_of_a_block_begins_with_the_same_tile(B, L, D):
    """A block's first ticket and its second go through the same word: more tiles than blocks that run, other kernels
    between, the same bits every time."""
    r = rng(80, B, L)
    g = Glr(r, B, L, D, "bf16")
    dy, dh0 = draw(r, (B, L, D), "bf16")[0], draw(r, (B, D), "fp32")[0]
    cfg = g.cfg(B, L)
    kept, other = kept_of(cfg), torch.empty(1 << 20, device="cuda")
    want = None
    for turn in range(60):
        y, h, dh = torch.zeros_like(g.x), torch.zeros_like(g.h), dh0.clone()
        if turn % 3:
            other.fill_(turn)
        g.forward(cfg, y, h, kept)
        o = [y, h, dh, *g.backward(cfg, dy, dh, kept).values()]
        if want is None:
            want = o
            for b in (0, B - 1):
                close(y[b], g.ref(b, g.hh[b])["y"], g.ref(b, g.hh[b], mag=True)["y"], "bf16", L, "y")
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_no_sequences():
    """A packed batch without sequences has no rows of theirs: nothing is read or written but the parameters' gradients,
    which are zeros."""
    D = 40
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = Glr(rng(81), 1, 0, D, "fp32", packed_rows=300)
    cfg = g.cfg(0, 300, seq_start=start)
    y = torch.full_like(g.x, 5.0)
    g.forward(cfg, y)
    o = g.backward(cfg, torch.ones_like(g.x), None)
    assert (y == 5).all() and all((o[k] == 7).all() for k in ("dx", "dr", "di", "dz"))
    assert not any(o[k].any() for k in ("dlam", "drb", "dib"))


def spread_like(got, want, what):
    """NaN in the places where the recurrence, token by token, has NaN, and nowhere else."""
    got, want = np.isnan(host(got)), np.isnan(want)
    assert (got == want).all(), f"{what}: {int((got & ~want).sum())} too many, {int((want & ~got).sum())} lost"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,lens", [(64, [1300, 1300, 1300]), (33, [90, 1400, 200]), (8, [4000]), (1024, [640] * 10)], ids=str)
def test_nan_reaches_the_rest_of_its_sequence(lens, D, dtype):
    """Decays of e^-1 to e^-200 a token, whose products over a warp's, a tile's or a group's rows leave the range: a NaN of
    one token is in all later states and outputs, and one of a gradient in those of all earlier tokens."""
    even, B = len(set(lens)) == 1, len(lens)
    r = rng(82, D, B)
    start, rows, at = packed(lens, 0)
    g = Glr(r, B, lens[0], D, dtype, **({} if even else dict(packed_rows=rows)))
    g.lam = dev(np.resize([0.5, 2.0, 5.0, 25.0, -6.0], D))
    g.lamh = host(g.lam)
    shape = tuple(g.x.shape)
    (dy, dyh), (dh, dhh) = draw(r, shape, dtype), draw(r, (B, D), "fp32")
    pick = (lambda b, t: (b, t)) if even else (lambda b, t: (at[b] + t,))
    seq = (lambda b: b) if even else (lambda b: slice(at[b], at[b] + lens[b]))
    b, n = B // 2, lens[B // 2]
    g.x[pick(b, 5)], g.xh[pick(b, 5)] = float("nan"), np.nan
    dy[pick(b, n - 3)], dyh[pick(b, n - 3)] = float("nan"), np.nan
    cfg = g.cfg(B, lens[0] if even else rows, **({} if even else dict(seq_start=start)))
    y, out, kept = torch.empty_like(g.x), torch.empty_like(g.h), kept_of(cfg)
    g.forward(cfg, y, out, kept)
    o = g.backward(cfg, dy, dh, kept)
    for i in range(B):
        with np.errstate(all="ignore"):
            ref = g.ref(seq(i), g.hh[i], dyh[seq(i)], dhh[i])
        spread_like(y[seq(i)], ref["y"], "y")
        spread_like(out[i], ref["h"], "h")
        spread_like(dh[i], ref["dh"], "dh")
        for k in ("dx", "dr", "di", "dz"):
            spread_like(o[k][seq(i)], ref[k], k)
    for k in ("dlam", "drb", "dib"):
        assert torch.isnan(o[k]).all(), k


def test_nan_stays_in_a_state_token_by_token():
    """Single tokens whose factor underflows: a state of NaN stays, one of zeros takes the token's input."""
    D, B = 40, 4
    g = Glr(rng(83), B, 1, D, "fp32", bias=False)
    g.lam.fill_(300.0)
    g.r.fill_(2.0)
    g.h[1], g.h[2, ::3] = float("nan"), float("nan")
    y, out = torch.empty_like(g.x), torch.empty_like(g.h)
    g.forward(g.cfg(B, 1), y, out)
    assert torch.equal(torch.isnan(out), torch.isnan(g.h)) and torch.equal(torch.isnan(y[:, 0]), torch.isnan(g.h))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rate", [-6.0, 2.0, 25.0])
@pytest.mark.parametrize("D,L", [(64, 1300), (33, 300), (8, 4000)])
def test_an_infinite_state_is_never_finite_again(D, L, rate, dtype):
    """Infinite inputs, first states and gradients: what is not finite token by token is not finite here (NaN, where the
    recurrence says infinity, is allowed), and nothing else."""
    B = 3
    r = rng(84, D, L)
    g = Glr(r, B, L, D, dtype)
    g.lam.fill_(rate)
    g.lamh = host(g.lam)
    (dy, dyh), (dh, dhh) = draw(r, (B, L, D), dtype), draw(r, (B, D), "fp32")
    inf = float("inf")
    g.x[0, 40], g.xh[0, 40] = inf, inf
    g.h[1], g.hh[1] = -inf, -inf
    dy[0, L - 30], dyh[0, L - 30] = -inf, -inf
    dh[2], dhh[2] = inf, inf
    cfg = g.cfg(B, L)
    y, out, kept = torch.empty_like(g.x), torch.empty_like(g.h), kept_of(cfg)
    g.forward(cfg, y, out, kept)
    o = g.backward(cfg, dy, dh, kept)
    for b in range(B):
        with np.errstate(all="ignore"):
            ref = g.ref(b, g.hh[b], dyh[b], dhh[b])
        for k, got in (("y", y[b]), ("h", out[b]), ("dh", dh[b]), *((k, o[k][b]) for k in ("dx", "dr", "di", "dz"))):
            assert (np.isfinite(host(got)) == np.isfinite(ref[k])).all(), (b, k)


def test_a_token_of_the_most_channels():
    """2^31 - 256 channels: the last ones are as they are alone."""
    D, n = 2 ** 31 - 256, 1000
    r = rng(85)
    tail = {k: dev(r.standard_normal(n), "bf16") for k in ("x", "r")}
    lam, h = dev(r.uniform(-6, 1, n)), dev(r.standard_normal(n))

    def padded(v):
        t = torch.zeros(1, D, device="cuda", dtype=v.dtype)
        t[0, -n:] = v
        return t
    outs = []
    for D_, lay in ((D, padded), (n, lambda v: v[None])):
        cfg = A.make_glr_cfg(1, 1, D_, c=C)
        y, out = lay(torch.zeros_like(tail["x"])), lay(h)
        A.atlas_glr_forward(lay(tail["x"]), lay(tail["r"]), None, None, lay(lam)[0], None, None, cfg, y, out, out)
        outs.append((y[0, -n:].clone(), out[0, -n:].clone()))
        del y, out
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[0][0].abs().max() > 0.1


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("D", [40, 33])
@pytest.mark.parametrize("start,good", [([0, 100, 50, 300], [0]), ([0, 100, 200, 301], [0, 1]), ([-1, 100, 200, 300], [1, 2]),
                                        ([0, 290, 300, 2 ** 31 - 1], [0, 1]), ([5, 2, 7, 300], [])], ids=str)
def test_gradients_beside_a_bad_sequence(start, good, D, keep):
    """A seq_start that falls, ends behind the rows or begins in front of them: the other sequences' gradients are theirs, the
    rows of those left out stay as they were, and nothing of them is in the parameters' gradients."""
    rows, B = 300, 3
    r = rng(86, D)
    g = Glr(r, B, 0, D, "fp32", packed_rows=rows)
    (dy, dyh), (dh, dhh) = draw(r, (rows, D), "fp32"), draw(r, (B, D), "fp32")
    before, st = dh.clone(), status()
    cfg = g.cfg(B, rows, seq_start=torch.tensor(start, dtype=torch.int32, device="cuda"), status_dev=st)
    kept = kept_of(cfg) if keep else None
    y, out = torch.full_like(g.x, 5.0), torch.full_like(g.h, 5.0)
    g.forward(cfg, y, out, kept)
    assert int(st) == A.ERR_INVALID
    st.zero_()
    o = g.backward(cfg, dy, dh, kept)
    assert int(st) == A.ERR_INVALID
    at = {b: slice(start[b], start[b + 1]) for b in good}
    # (check_grads adds up the good ones' sums; dh by their numbers)
    check_grads(g, o, dh, [(at[b], b, start[b + 1] - start[b]) for b in good], dyh, dhh)
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    for b in good:
        left[at[b]] = False
        close(y[at[b]], g.ref(at[b], g.hh[b])["y"], g.ref(at[b], g.hh[b], mag=True)["y"], "fp32", rows, "y")
    assert (y[left] == 5).all()
    for k in ("dx", "dr", "di", "dz"):
        assert (o[k][left] == 7).all(), k
    for b in range(B):
        if b not in good:
            assert torch.equal(dh[b], before[b]) and (out[b] == 5).all()


def test_the_longest_sequence():
    """2^31 - 1 tokens of one channel, decays that forget within a few hundred: the last states, outputs and gradients are those
    of the last tokens alone, the first gradients those of the first."""
    L, n = 2 ** 31 - 1, 4096
    lam = torch.full((1,), -1.0, device="cuda")
    r = rng(87)
    parts = {k: dev(r.standard_normal((2, n, 1)), "bf16") for k in ("x", "r", "dy")}

    def whole(k):
        t = torch.zeros(1, L, 1, device="cuda", dtype=torch.bfloat16)
        t[0, :n], t[0, -n:] = parts[k][0], parts[k][1]
        return t

    def run(x, rr, dy, length):
        cfg = A.make_glr_cfg(1, length, 1, c=C)
        space(cfg, max(A.atlas_glr_workspace_bytes(cfg), A.atlas_glr_backward_workspace_bytes(cfg)))
        y, h, kept = torch.empty_like(x), torch.empty(1, 1, device="cuda"), kept_of(cfg)
        A.atlas_glr_forward(x, rr, None, None, lam, None, None, cfg, y, None, h, kept)
        ends = [y[0, :n].clone(), y[0, -n:].clone(), h.clone()]
        dx, dr, dlam = y, torch.empty_like(x), torch.empty_like(lam)  # (y has been read)
        A.atlas_glr_backward(x, rr, None, None, lam, None, None, cfg, None, kept, dy, None, dx, dr, None, None, dlam, None, None)
        return ends + [dx[0, :n].clone(), dx[0, -n:].clone(), dr[0, :n].clone(), dr[0, -n:].clone()], dlam.clone()
    got, dlam = run(whole("x"), whole("r"), whole("dy"), L)
    first, last = ([p[k][i:i + 1].contiguous() for k in ("x", "r", "dy")] for i, p in ((0, parts), (1, parts)))
    (a, da), (b, db) = run(*first, n), run(*last, n)
    # (the first part ends in zeros here and in nothing there, the last one begins with a state that has decayed to nothing)
    for k, (g, want) in enumerate(zip(got, (a[0], b[1], b[2], a[3], b[4], a[5], b[6]))):
        cut = slice(0, n - 600) if k in (3, 5) else slice(None)  # the first part's gradients
        assert (g[cut].float() - want[cut].float()).abs().max() <= 2.0 ** -7 * want.float().abs().max(), k
        # (the last state is one number, a h + sqrt(1 - a^2) x of normal ones: it may be any small one)
        assert want.float().abs().max() > (0.1 if want.numel() > 1 else 0), k
    assert (dlam - da - db).abs() <= 2.0 ** -12 * (da.abs() + db.abs())
