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
