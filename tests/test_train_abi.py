"""CPU-only checks of the cross-entropy and Newton-Schulz entry points: sizes of
the workspaces, and what they refuse before touching a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_exact_attention_ra_gb300 as ra
    return ra


VP = ctypes.c_void_p(4096)
BIG = ctypes.c_size_t(1 << 50)


def test_xent_workspaces(ra):
    fwd, bwd = ra.ra_xent_fwd_workspace_bytes, ra.ra_xent_bwd_workspace_bytes
    assert fwd(ra.RA_BF16, 1000, 64, 3001) >= 1000 * 4 + 1000 * 8 * ((3001 + 127) // 128)
    assert fwd(ra.RA_F32, 1000, 64, 3001) == 0 and fwd(ra.RA_BF16, 0, 64, 10) == 0
    T, V = 100000, 3001
    one = bwd(ra.RA_BF16, ra.RA_BF16, T, 64, V, V)
    assert one >= T * V * 2
    assert bwd(ra.RA_BF16, ra.RA_BF16, T, 64, V, 1 << 30) == one      # a block past V is V
    some = bwd(ra.RA_BF16, ra.RA_BF16, T, 64, V, 512)
    assert T * (512 * 2 + 64 * 4) <= some < one
    assert bwd(ra.RA_BF16, ra.RA_F32, T, 64, V, 512) <= some - T * 64 * 4
    assert bwd(ra.RA_BF16, 9, T, 64, V, 512) == 0
    # a narrow block is widened until its gradient takes 256 MB
    assert bwd(ra.RA_BF16, ra.RA_F32, 1000, 64, V, 1) == bwd(ra.RA_BF16, ra.RA_F32, 1000, 64, V, V)


def test_xent_refusals(ra):
    lib = ra.lib

    def fwd(*, dtype=ra.RA_BF16, T=100, D=64, V=300, xs=0, ws=0, x=VP, w=VP, y=VP, loss=VP, lse=VP, wsp=VP, n=BIG):
        return lib.ra_xent_fwd(x, w, dtype, T, D, V, xs, ws, y, -100, loss, lse, wsp, n, None)

    def bwd(*, dtype=ra.RA_BF16, T=100, D=64, V=300, xs=0, ws=0, y=VP, lse=VP, g=VP, block=128, dx=VP, dxt=ra.RA_F32,
            dw=VP, dwt=ra.RA_F32, wsp=VP, n=BIG):
        return lib.ra_xent_bwd(VP, VP, dtype, T, D, V, xs, ws, y, -100, lse, g, block, dx, dxt, dw, dwt, wsp, n, None)

    for call in (fwd, bwd):
        assert call(dtype=ra.RA_F32) == 2
        assert call(T=0) == 1 and call(V=0) == 1 and call(D=0) == 1 and call(T=-5) == 1
        assert call(D=60) == 2 and "multiple of 8" in ra.ra_last_error()
        assert call(xs=56) == 1 and call(ws=32) == 1 and "stride" in ra.ra_last_error()
        assert call(xs=68) == 1 and call(ws=100) == 1
        assert call(T=1 << 31) == 1 and call(V=(1 << 30) + 1) == 1
        assert call(y=None) == 1 and "targets" in ra.ra_last_error()
        assert call(y=ctypes.c_void_p(4100)) == 1
        assert call(wsp=None) == 1 and call(n=ctypes.c_size_t(64)) == 1 and "workspace" in ra.ra_last_error()
        assert call(wsp=ctypes.c_void_p(4096 + 64)) == 1 and "aligned" in ra.ra_last_error()
        assert call(lse=None) == 1 and "lse" in ra.ra_last_error()
    assert fwd(x=None) == 1 and fwd(w=ctypes.c_void_p(4104)) == 1
    assert fwd(loss=None) == 1 and "loss" in ra.ra_last_error()
    assert bwd(g=None) == 1 and "dloss" in ra.ra_last_error()
    assert bwd(block=0) == 1 and bwd(dxt=7) == 1 and bwd(dwt=-1) == 1
    assert bwd(dx=None) == 1 and bwd(dw=ctypes.c_void_p(4100)) == 1


def test_newton_schulz_workspace(ra):
    size = ra.ra_newton_schulz_workspace_bytes
    assert size(1, 1000, 333) >= 3 * 2 * 1000 * 333 + 2 * 2 * 333 * 333
    assert size(4, 1000, 333) > 3.9 * size(1, 1000, 333)
    assert size(0, 10, 10) == 0 and size(1, 10, 70000) == 0 and size(1, -1, 10) == 0


def test_newton_schulz_refusals(ra):
    lib = ra.lib

    def call(*, g=VP, dt=ra.RA_F32, batch=2, rows=40, cols=50, gb=0, gr=0, co=(3.4445, -4.775, 2.0315), steps=5, eps=1e-7,
             out=VP, odt=ra.RA_BF16, ob=0, orr=0, wsp=VP, n=BIG):
        c = None if co is None else (ctypes.c_float * 3)(*co)
        return lib.ra_newton_schulz(g, dt, batch, rows, cols, gb, gr, c, steps, eps, out, odt, ob, orr, wsp, n, None)

    assert call(batch=0) == 1 and call(rows=0) == 1 and call(cols=-3) == 1 and call(steps=0) == 1
    assert call(rows=65537) == 1 and call(steps=101) == 1
    assert call(co=None) == 1 and call(co=(float("nan"), 0, 0)) == 1 and call(co=(1, float("inf"), 0)) == 1
    assert call(co=(8.0, 1.0, 1.0)) == 2 and "singular" in ra.ra_last_error()
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(dt=5) == 1 and call(odt=-1) == 1
    assert call(g=None) == 1 and call(out=ctypes.c_void_p(4097)) == 1 and "out" in ra.ra_last_error()
    assert call(gr=49) == 1 and call(gb=100) == 1 and call(orr=20) == 1 and call(ob=-1) == 1
    assert "stride" in ra.ra_last_error()
    assert call(wsp=None) == 1 and call(n=ctypes.c_size_t(1000)) == 1 and "workspace" in ra.ra_last_error()
    assert call(wsp=ctypes.c_void_p(4096 + 128)) == 1


def test_binding_refuses_before_the_library(ra):
    x, w, y = torch.zeros(4, 16).bfloat16(), torch.zeros(9, 16).bfloat16(), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    for bad in (lambda: ra.xent_fwd(x, w[:, :8], y), lambda: ra.xent_fwd(x, w.half(), y),
                lambda: ra.xent_fwd(x, w, y.int()), lambda: ra.xent_fwd(x, w, y[:3]),
                lambda: ra.xent_fwd(x[0], w, y), lambda: ra.xent_fwd(x.T.contiguous().T, w, y),
                lambda: ra.ra_xent_fwd(x, w, y, f, f[:3], f), lambda: ra.ra_xent_fwd(x, w, y, f, f.double(), f),
                lambda: ra.ra_xent_bwd(x, w, y, f, f, 4, x.T, w, f), lambda: ra.ra_xent_bwd(x, w, y, f, f, 4, x, w[:4], f),
                lambda: ra.newton_schulz(torch.zeros(3)), lambda: ra.newton_schulz(torch.zeros(4, 6).T),
                lambda: ra.ra_newton_schulz(torch.zeros(4, 6), torch.zeros(6, 4), f),
                # tensors that are not on the current device
                lambda: ra.ra_xent_fwd(x, w, y, f, f, f), lambda: ra.ra_newton_schulz(x, x, f)):
        with pytest.raises(ra.RAError):
            bad()


def test_binding_refuses_expanded_tensors(ra):
    """A stride of 0 means packed to the library: an expanded tensor would be read past its end."""
    x, w, y = torch.zeros(4, 16).bfloat16(), torch.zeros(9, 16).bfloat16(), torch.zeros(4, dtype=torch.int64)
    f, g = torch.zeros(4), torch.zeros(2, 4, 6)
    for bad in (lambda: ra.xent_fwd(x[:1].expand(4, 16), w, y), lambda: ra.xent_fwd(x, w[:1].expand(9, 16), y),
                lambda: ra.xent_bwd(x[:1].expand(4, 16), w, y, f, f), lambda: ra.newton_schulz(g[:1].expand(2, 4, 6)),
                lambda: ra.newton_schulz(g[:, :1].expand(2, 4, 6)), lambda: ra.newton_schulz(g[0, :1].expand(4, 6)),
                lambda: ra.ra_newton_schulz(g, g[:1].expand(2, 4, 6), f)):
        with pytest.raises(ra.RAError, match="expanded"):
            bad()
