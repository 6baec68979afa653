"""The first call of a process is captured into a graph: kernels that are loaded and asked for their registers there."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """if True:
    import torch
    import test_memorization_recurrent_gb300 as A
    what, rows, d = {what!r}, {rows}, {d}
    torch.manual_seed(0)
    t = [torch.randn(rows, d, device="cuda").bfloat16() for _ in range(5)]
    p = [torch.randn(d, device="cuda") - 4 for _ in range(2)]
    w = torch.randn(d, device="cuda").bfloat16()
    out = [torch.empty_like(t[0]) for _ in range(6)] + [torch.empty(d, device="cuda") for _ in range(3)]
    if what == "layernorm":
        cfg = A.make_norm_cfg(rows, d, eps=1e-5)
        ws = torch.empty(A.atlas_layernorm_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")

        def call():
            A.atlas_layernorm_forward(t[0], t[1], w, w, cfg, out[0], out[1])
            A.atlas_layernorm_backward(t[0], w, t[2], t[3], cfg, out[2], out[6], out[7])
    else:
        cfg = A.make_glr_cfg(1, rows, d)
        ws = torch.empty(A.atlas_glr_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")

        def call():
            A.atlas_glr_forward(t[0], t[1], t[2], t[3], p[0], None, None, cfg, out[0])
            A.atlas_glr_backward(t[0], t[1], t[2], t[3], p[0], None, None, cfg, None, None, t[4], None, *out[1:5], out[6], None, None)
    cfg.workspace, cfg.workspace_bytes, cfg.held = ws.data_ptr(), ws.numel(), (ws,)
    used = out[:3] + out[6:8] if what == "layernorm" else out[:5] + out[6:7]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in used]
    for o in used:
        o.zero_()
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, used)) and all(o.float().abs().sum() > 0 for o in got)
    print("equal")
"""


@pytest.mark.parametrize("what,rows,d", [("layernorm", 2000, 128), ("layernorm", 2000, 1371), ("layernorm", 20, 2048), ("layernorm", 200, 9001),
                                         ("glr", 3000, 96), ("glr", 300, 33)])
def test_the_first_call_is_captured(what, rows, d):
    from test_memorization_recurrent_gb300 import build
    build.build()
    run = subprocess.run([sys.executable, "-c", CODE.format(what=what, rows=rows, d=d)], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]
