"""The gated linear recurrence without a GPU: descriptions at the ends of their ranges."""
import pytest

import test_memorization_recurrent_gb300 as A
from test_memorization_recurrent_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return A.load_library()


def test_rows_without_sequences_are_none(lib):
    """A packed batch of no sequences keeps no states, whatever its rows (seq_start has one element, and no tile may look
    for a row's sequence)."""
    for L in (0, 1, 300, 10 ** 6):
        cfg = A.make_glr_cfg(0, L, 40, seq_start=16)
        assert A.atlas_glr_kept_bytes(cfg) == A.atlas_glr_kept_bytes(A.make_glr_cfg(0, L, 40)) == 0
        assert A.atlas_glr_backward_workspace_bytes(cfg) < 4096
    assert A.atlas_glr_kept_bytes(A.make_glr_cfg(1, 300, 40, seq_start=16)) == 3 * 40 * 4
