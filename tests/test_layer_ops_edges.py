"""Layer operators without a GPU: sizes of workspaces."""
import pytest

import test_memorization_recurrent_gb300 as A
from test_memorization_recurrent_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.mark.parametrize("B,L,D,N", [(1000, 10000, 2048, 16), (64, 200, 512, 16), (5, 100000, 64, 16), (4000, 4000, 64, 64), (300, 70000, 33, 7)])
def test_scan_backward_workspace_goes_by_rows(B, L, D, N):
    """A packed batch keeps a state every eight rows and one more a sequence, and a few a segment; segments
    have 128 tokens or more, and there is one more a sequence."""
    got = A.atlas_scan_backward_workspace_bytes(A.make_scan_cfg(B, L, D, N, seq_start=16))
    kept, segments, padded = L // 8 + B, L // 128 + B, 4 * max(2, 1 << (-(-N // 4) - 1).bit_length())
    blocks = -(-D // (256 // (padded // 4)))  # of the main pass, over channels
    most = 4 * D * ((N + 1) * kept + 3 * (N + 1) * segments) + 8 * padded * blocks * L + 256
    assert got <= most, (got, most)


def test_workspaces_of_lengths_next_to_2_to_the_31():
    """Segments of the longest sequences are counted, not wrapped: two states and a decay each."""
    for kw in (dict(B=1), dict(B=1, seq_start=16)):
        cfg = A.make_scan_cfg(L=2 ** 31 - 1, D=1, N=1, **kw)
        assert 0 < A.atlas_scan_workspace_bytes(cfg) < 1 << 20
        assert 0 < A.atlas_scan_backward_workspace_bytes(cfg) < 1 << 39
    assert 0 < A.atlas_conv_backward_workspace_bytes(A.make_conv_cfg(1, 2 ** 31 - 1, 1, 4)) < 1 << 20


def test_views_that_end_too_early_are_refused(monkeypatch):
    """An expanded or narrowed view may count more elements than its storage holds: what is checked is the
    storage from its first element on."""
    torch = pytest.importorskip("torch")
    from test_memorization_recurrent_gb300 import ops
    monkeypatch.setattr(ops, "_types", (torch.float32, torch.bfloat16, torch.float16))
    strided = 2 * 40  # 40 elements from the first to the last, not necessarily dense

    def ok(t):
        return ops._arg(t, A.F32, strided, "x", -1) == t.data_ptr()
    row = torch.zeros(8)
    wide = torch.zeros(5, 16)
    assert ok(torch.zeros(40)) and ok(wide[:, :8]) and ok(torch.zeros(8, 5).t())
    for bad in (row.expand(100, 8), row[:, None].expand(8, 100), torch.zeros(39), wide[3:, :8], torch.zeros(20, 2)[:, 0][1:], torch.zeros(10, 4)[4:].t()):
        with pytest.raises(A.AtlasError):
            ok(bad)


class OnDevice:
    """What the binding looks at of a tensor of a description."""

    def __init__(self, dtype, n, device):
        self.dtype, self.n, self.device, self.is_cuda = dtype, n, device, True

    def numel(self):
        return self.n

    def element_size(self):
        return 4

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 16

    def get_device(self):
        return self.device


def test_tensors_of_a_description_are_on_the_current_device(monkeypatch):
    torch = pytest.importorskip("torch")
    from test_memorization_recurrent_gb300 import ops
    launched = []
    monkeypatch.setattr(ops, "_types", (torch.float32, torch.bfloat16, torch.float16))
    monkeypatch.setattr(ops, "_fn", {name: lambda *a: launched.append(a) or 0 for name in A.OPS_EXPORTS})
    monkeypatch.setattr(ops, "_device", lambda: 0)
    i32 = torch.int32
    for device in (0, 1):
        start, slot, space = OnDevice(i32, 3, device), OnDevice(i32, 2, device), OnDevice(torch.float32, 64, device)
        cfgs = ((A.atlas_conv_forward, [16, 16, None], A.make_conv_cfg(2, 4, 8, 4, seq_start=start), [16]),
                (A.atlas_scan_forward, [16] * 5 + [None] * 3, A.make_scan_cfg(2, 4, 8, 4, slot=slot, n_slots=2), [16]),
                (A.atlas_norm_backward, [16, 16, 16, None], A.make_norm_cfg(2, 8, workspace=space, workspace_bytes=64), [16]))
        for f, before, cfg, after in cfgs:
            if device == 0:
                f(*before, cfg, *after, stream=0)
            else:
                with pytest.raises(A.AtlasError):
                    f(*before, cfg, *after, stream=0)
    assert len(launched) == 3
    with pytest.raises(A.AtlasError):  # not all on one device
        A.make_conv_cfg(2, 4, 8, 4, seq_start=OnDevice(i32, 3, 0), slot=OnDevice(i32, 2, 1), n_slots=2)


@pytest.mark.parametrize("bad", [4, 9, -1])
def test_unknown_element_types_are_refused_by_the_calls(monkeypatch, bad):
    torch = pytest.importorskip("torch")
    from test_memorization_recurrent_gb300 import ops
    monkeypatch.setattr(ops, "_types", (torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn))
    monkeypatch.setattr(ops, "_fn", {name: lambda *a: A.OK for name in A.OPS_EXPORTS})
    monkeypatch.setattr(ops, "_device", lambda: -1)
    x = torch.zeros(2, 8)
    for f, args, cfg in ((A.atlas_norm_forward, [x, None, None], A.make_norm_cfg(2, 8, dtype=bad)), (A.atlas_norm_forward, [x, None, None], A.make_norm_cfg(2, 8, dtype=A.F32, out_dtype=bad)),
                         (A.atlas_conv_forward, [x, x, None], A.make_conv_cfg(1, 2, 8, 2, dtype=A.F32, w_dtype=bad)), (A.atlas_scan_forward, [x] * 5 + [None] * 3, A.make_scan_cfg(1, 2, 8, 1, dtype=bad))):
        with pytest.raises(A.AtlasError):
            f(*args, cfg, x, stream=0)
