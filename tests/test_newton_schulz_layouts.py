"""Matrices of a batch whose rows lie between each other's, as the heads of a fused projection's
gradient [rows, heads, cols] do: they do not overlap, so they need no copy."""
import ctypes
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_exact_attention_ra_gb300 as ra
    return ra


@pytest.mark.parametrize("bs,rs,fits", [
    (2000, 50, True), (1999, 50, False),        # one matrix after the other
    (50, 150, True), (50, 149, False), (49, 150, False), (60, 170, True), (60, 169, False),  # rows between rows
    (50, 50, False),
])
def test_which_strides_are_taken(ra, bs, rs, fits):
    """40 x 50 matrices, 3 of them: what the library says of the strides, before it looks at the
    workspace (too small here)."""
    vp = ctypes.c_void_p(4096)
    for sides in ((bs, rs, 0, 0), (0, 0, bs, rs)):
        g_bs, g_rs, out_bs, out_rs = sides
        assert ra.lib.ra_newton_schulz(vp, ra.RA_F32, 3, 40, 50, g_bs, g_rs, (ctypes.c_float * 3)(1.5, -0.5, 0.0), 5, 1e-7,
                                       vp, ra.RA_F32, out_bs, out_rs, vp, ctypes.c_size_t(8), None) == 1
        assert ("workspace" if fits else "overlap") in ra.ra_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(100, 77), (64, 96), (150, 177), (200, 264), (77, 300), (300, 129)])
def test_matrices_whose_rows_lie_between_each_others(ra, rows, cols):
    from tests.test_gpu_newton_schulz import gradient
    g = gradient(rows, cols, 71, batch=3)
    want = ra.newton_schulz(g)
    wide = torch.full((rows, 4, cols), float("nan"), device="cuda")   # the last one belongs to nobody
    view = wide.permute(1, 0, 2)[:3]
    view.copy_(g)
    assert torch.equal(ra.newton_schulz(view), want)
    ws = torch.empty(ra.ra_newton_schulz_workspace_bytes(3, rows, cols), dtype=torch.uint8, device="cuda")
    ra.ra_newton_schulz(view, view, ws)         # in place
    ra.ra_sync_status()
    assert torch.equal(view, want) and torch.isnan(wide[:, 3]).all()
