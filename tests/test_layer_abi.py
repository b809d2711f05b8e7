"""CPU-only checks of the rotary, norm and clipping entry points: the frequencies, the sizes
of the workspaces, and what they refuse before touching a GPU."""
import ctypes
import math

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


def test_frequencies(ra):
    f = ra.rotary_frequencies(16, 1000.0, device="cpu")
    assert torch.allclose(f, torch.tensor([1000.0 ** (-i / 8) for i in range(8)], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(ra.rotary_frequencies(16, 1000.0, 4.0, device="cpu"), f / 4)
    b = ra.rotary_frequencies(16, 1000.0, 4.0, "base", device="cpu")
    assert b[0] == 1 and float(b[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-14)
    p = ra.rotary_frequencies(16, 1000.0, 4.0, "parts", trained=2000, fast=32, slow=1, device="cpu")
    for x, y in zip(f.tolist(), p.tolist()):
        turns = 2000 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert y == pytest.approx(x * (keep + (1 - keep) / 4), rel=1e-13)
    assert p[0] == f[0] and float(p[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-13)
    assert torch.equal(ra.rotary_frequencies(16, 1000.0, 1.0, "parts", trained=2000, device="cpu"), f)
    for bad in (dict(rot=0), dict(rot=7), dict(rot=258), dict(rot=8, base=1.0), dict(rot=8, base=math.inf),
                dict(rot=8, scale=0.5), dict(rot=8, scale=math.nan), dict(rot=2, method="base"),
                dict(rot=8, method="parts"), dict(rot=8, method="parts", trained=100, fast=1, slow=1),
                dict(rot=8, method="other")):
        with pytest.raises(ra.RAError):
            ra.rotary_frequencies(device="cpu", **bad)
    with pytest.raises(ra.RAError):
        ra.ra_rotary_frequencies(8, 10.0, 1, 0, 0, 0, 0, torch.empty(4))


def shape(ra, **kw):
    d = dict(B=2, N_q=8, N_kv=8, Hq=4, Hkv=2, d=64)
    d.update(kw)
    return ra.RaShape(*[d.get(n, 0) for n, _ in ra.RaShape._fields_])


def rotary(ra, **kw):
    d = dict(rot=64, freq=4096, positions=None, pos_bstride=0, pos_off=0, P=1, amplitude=1.0)
    d.update(kw)
    return ra.RaRotary(*[d[n] for n, _ in ra.RaRotary._fields_])


def test_rotary_refusals(ra):
    lib = ra.lib

    def plain(*, q=VP, k=VP, dt=ra.RA_BF16, sh=None, rot=None, flags=0, qo=VP, ko=VP, osh=None, **kw):
        sh = sh or shape(ra, **kw)
        return lib.ra_rotary_fwd(q, k, dt, sh, rot or rotary(ra), flags, qo, ko, osh or sh, None)

    def back(*, q=VP, k=VP, dt=ra.RA_BF16, sh=None, rot=None, flags=0, qo=VP, ko=VP, osh=None, gdt=None, **kw):
        sh = sh or shape(ra, **kw)
        return lib.ra_rotary_bwd(q, k, dt, sh, rot or rotary(ra), flags, qo, ko, dt if gdt is None else gdt, osh or sh, None)

    def norm(*, q=VP, k=VP, dt=ra.RA_BF16, sh=None, rot=None, flags=0, qo=VP, ko=VP, osh=None, qw=VP, kw=VP, wdt=0, eps=1e-6, **more):
        sh = sh or shape(ra, **more)
        return lib.ra_norm_rotary_fwd(q, k, dt, sh, qw, kw, wdt, eps, rot or rotary(ra), flags, qo, ko, osh or sh, None)

    def norm_back(*, q=VP, k=VP, dt=ra.RA_BF16, sh=None, rot=None, flags=0, qo=VP, ko=VP, osh=None, qw=VP, kw=VP, wdt=0,
                  eps=1e-6, dqo=VP, dko=VP, ddt=None, dsh=None, gdt=None, dqw=VP, dkw=VP, ws=VP, n=BIG, **more):
        sh = sh or shape(ra, **more)
        return lib.ra_norm_rotary_bwd(q, k, dt, sh, dqo, dko, dt if ddt is None else ddt, dsh or sh, qw, kw, wdt, eps,
                                      rot or rotary(ra), flags, qo, ko, dt if gdt is None else gdt, osh or sh, dqw, dkw, ws,
                                      n, None)

    for call in (plain, back, norm, norm_back):
        assert call(B=0) == 1 and call(Hq=3) == 1 and call(N_kv=9) == 1 and "rows" in ra.ra_last_error()
        assert call(d=60) == 2 and call(d=264, rot=rotary(ra, rot=0)) == 2 and "multiple of 8" in ra.ra_last_error()
        assert call(dt=5) == 1 and call(flags=1) == 1 and call(flags=16) == 1
        assert call(rot=rotary(ra, rot=7)) == 1 and call(rot=rotary(ra, rot=66)) == 1 and call(rot=rotary(ra, rot=-2)) == 1
        assert call(rot=rotary(ra, freq=None)) == 1 and call(rot=rotary(ra, freq=4100)) == 1 and "freq" in ra.ra_last_error()
        assert call(rot=rotary(ra, positions=4100)) == 1 and call(rot=rotary(ra, positions=4096, pos_bstride=7)) == 1
        assert call(rot=rotary(ra, positions=4096), flags=ra.RA_STRIPED) == 1
        assert call(rot=rotary(ra, P=3), flags=ra.RA_STRIPED) == 1 and call(rot=rotary(ra, P=0), flags=ra.RA_STRIPED) == 1
        assert call(rot=rotary(ra, amplitude=math.inf)) == 1 and call(rot=rotary(ra, amplitude=math.nan)) == 1
        assert call(q=None) == 1 and call(q=ctypes.c_void_p(4104)) == 1 and call(qo=None) == 1
        assert call(k=None) == 1 and call(ko=None) == 1 and call(ko=ctypes.c_void_p(8)) == 1
        assert call(q_rstride=260) == 1 and "16 bytes" in ra.ra_last_error()
        assert call(osh=shape(ra, N_q=7)) == 1 and call(osh=shape(ra, q_hstride=65)) == 1
        assert call(q_hstride=32) == 1 and call(kv_bstride=100) == 1
    assert back(gdt=ra.RA_F32) == 2 and back(dt=ra.RA_F32, gdt=9) == 1
    for call in (norm, norm_back):
        assert call(eps=-1.0) == 1 and call(eps=math.nan) == 1 and call(wdt=7) == 1 and call(qw=ctypes.c_void_p(4098)) == 1
    assert norm_back(ddt=ra.RA_F16) == 2 and norm_back(gdt=ra.RA_F16) == 2
    assert norm_back(dqo=None) == 1 and norm_back(dko=None) == 1 and norm_back(dsh=shape(ra, d=32)) == 1
    assert norm_back(dqw=ctypes.c_void_p(4098)) == 1 and norm_back(dkw=ctypes.c_void_p(4098)) == 1
    assert norm_back(k=None, dko=None, ko=None) == 1 and "dk_weight" in ra.ra_last_error()
    assert norm_back(ws=None) == 1 and norm_back(n=ctypes.c_size_t(100)) == 1 and norm_back(ws=ctypes.c_void_p(4224)) == 1
    size = ra.ra_norm_rotary_bwd_workspace_bytes
    assert size(0) == 0 and size(257) == 0 and size(128) == 2 * size(64) > 0


def test_clip_refusals(ra):
    lib = ra.lib

    def arrays(addresses, sizes, types):
        n = len(sizes)
        return (ctypes.c_void_p * n)(*addresses), (ctypes.c_longlong * n)(*sizes), (ctypes.c_int * n)(*types)

    def clip(addresses=(4096, 8192), sizes=(10, 20), types=(0, 1), outs=None, out_types=(0, 1), max_norm=1.0, eps=1e-6,
             norm=VP, ws=VP, n=BIG, count=None):
        g, s, t = arrays(addresses, sizes, types)
        o = ot = None
        if outs is not None:
            o, _, ot = arrays(outs, sizes, out_types)
        return lib.ra_grad_clip(g, s, t, len(sizes) if count is None else count, max_norm, eps, o, ot, norm, ws, n, None)

    def norm(addresses=(4096, 8192), sizes=(10, 20), types=(0, 1), norm=VP, ws=VP, n=BIG, count=None):
        return lib.ra_grad_norm(*arrays(addresses, sizes, types), len(sizes) if count is None else count, norm, ws, n, None)

    for call in (clip, norm):
        assert call(count=0) == 1 and call(count=-1) == 1 and call(count=(1 << 20) + 1) == 1
        assert call(types=(0, 3)) == 1 and call(sizes=(-1, 2)) == 1 and call(sizes=(1 << 41, 2)) == 1
        assert call(sizes=(1 << 40, 1 << 40)) == 1
        assert call(addresses=(None, 8192)) == 1 and call(addresses=(4098, 8192)) == 1 and call(addresses=(4096, 8193)) == 1
        assert call(norm=None) == 1 and call(norm=ctypes.c_void_p(4098)) == 1
        assert call(ws=None) == 1 and call(n=ctypes.c_size_t(64)) == 1 and call(ws=ctypes.c_void_p(4096 + 128)) == 1
    assert clip(max_norm=-1.0) == 1 and clip(max_norm=math.inf) == 1 and clip(max_norm=math.nan) == 1 and clip(eps=-1.0) == 1
    assert clip(outs=(None, 8192)) == 1 and clip(outs=(4096, 8192), out_types=(0, 8)) == 1
    # no output overlaps another tensor
    assert clip(addresses=(4096, 4096), types=(0, 0)) == 1 and "overlap" in ra.ra_last_error()
    assert clip(addresses=(4096, 4096 + 36), types=(0, 0)) == 1                          # in place, one element shared
    assert clip(outs=(16384, 16384 + 36)) == 1                                           # two outputs
    assert clip(outs=(8192 + 36, 65536)) == 1 and "overlaps" in ra.ra_last_error()       # an output and another's input
    assert clip(outs=(4100, 65536)) == 1 and clip(outs=(4096, 65536), out_types=(1, 1)) == 1  # its own, not in place
    assert ra.ra_grad_workspace_bytes(0) == 0 and ra.ra_grad_workspace_bytes(1 << 21) == 0
    assert ra.ra_grad_workspace_bytes(1) > 0 and ra.ra_grad_workspace_bytes(1025) == 2 * ra.ra_grad_workspace_bytes(1024)


def test_cross_refusals(ra):
    lib = ra.lib

    def fwd(*, q=VP, k=VP, v=VP, dt=ra.RA_BF16, sh=None, lens=None, flags=0, scale=0.1, o=VP, odt=ra.RA_F32, lse=VP, ws=VP,
            n=BIG, **kw):
        return lib.ra_cross_fwd(q, k, v, dt, sh or shape(ra, **kw), lens, flags, scale, o, odt, lse, ws, n, None)

    def bwd(*, q=VP, k=VP, v=VP, dt=ra.RA_BF16, sh=None, lens=None, flags=0, scale=0.1, o=VP, odt=ra.RA_F32, lse=VP, ws=VP,
            n=BIG, do=VP, dq=VP, dk=VP, dv=VP, gdt=ra.RA_F32, **kw):
        return lib.ra_cross_bwd(q, k, v, o, odt, do, lse, dt, sh or shape(ra, **kw), lens, flags, scale, dq, dk, dv, gdt, ws, n,
                                None)

    for call in (fwd, bwd):
        for size in (dict(N_q=1, N_kv=70), dict(N_q=300, N_kv=7)):       # both kernels
            assert call(dt=ra.RA_F32, **size) == 2 and call(dt=7, **size) == 1 and call(odt=9, **size) == 1
            assert call(B=0, **size) == 1 and call(Hq=3, **size) == 1 and call(d=32, **size) == 2 and call(d=96, **size) == 2
            assert call(flags=1, **size) == 1 and call(flags=4, **size) == 1 and "flag" in ra.ra_last_error()
            assert call(scale=0.0, **size) == 1 and call(scale=math.nan, **size) == 1
            for name in ("q", "k", "v", "o"):
                assert call(**{name: None}, **size) == 1 and call(**{name: ctypes.c_void_p(4104)}, **size) == 1
            assert call(lse=None, **size) == 1 and call(lse=ctypes.c_void_p(4098), **size) == 1
            assert call(lens=ctypes.c_void_p(4098), **size) == 1 and "kv_len" in ra.ra_last_error()
            assert call(ws=None, **size) == 1 and call(n=ctypes.c_size_t(16), **size) == 1 and call(ws=ctypes.c_void_p(4224), **size) == 1
            assert call(q_hstride=32, **size) == 1 and call(kv_bstride=100, **size) == 1
        assert call(N_q=0) == 1 and call(N_kv=0) == 1
        assert call(N_q=(1 << 30) - 1, B=64, Hq=64) == 2 and "tiles" in ra.ra_last_error()
    for name in ("do", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == 1 and bwd(**{name: ctypes.c_void_p(8)}) == 1
    assert bwd(gdt=5) == 1
    f, b = ra.ra_cross_fwd_workspace_bytes, ra.ra_cross_bwd_workspace_bytes
    long = shape(ra, B=1, N_q=4096, N_kv=10000, Hq=8, Hkv=8, d=128)
    assert f(ra.RA_BF16, long) >= 10000 * 8 * 128 * 2 and f(ra.RA_F16, long) < f(ra.RA_BF16, long)
    one = shape(ra, B=1, N_q=1, N_kv=100000, Hq=8, Hkv=8, d=128)
    assert 8 * 128 * 4 * 8 < f(ra.RA_BF16, one) < 1 << 22           # parts' states, no copy of v
    assert f(ra.RA_F32, long) == 0 and b(ra.RA_F32, long) == 0 and f(ra.RA_BF16, shape(ra, d=32)) == 0
    assert b(ra.RA_BF16, long) >= 4096 * 8 * 128 * (4 + 2 + 2) + 2 * 10000 * 8 * 128 * 2


def test_cross_binding_refuses_before_the_library(ra):
    q, k = torch.zeros(2, 3, 4, 64).half(), torch.zeros(2, 9, 2, 64).half()
    lse, ws, n = torch.zeros(2, 4, 3), torch.zeros(64, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: ra.cross_attention_fwd(q[:1], k, k), lambda: ra.cross_attention_fwd(q, k.float(), k),
                lambda: ra.cross_attention_fwd(q, k, k.float()), lambda: ra.cross_attention_fwd(q, k, k[:, :8]),
                lambda: ra.cross_attention_fwd(q[..., :32], k, k), lambda: ra.cross_attention_fwd(q[0], k, k),
                lambda: ra.cross_attention_fwd(q, k, k.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: ra.cross_attention_fwd(q, k, k, n.long()), lambda: ra.cross_attention_fwd(q, k, k, n[:1]),
                lambda: ra.cross_attention_fwd(q, k, k, n.repeat(2)[::2]), lambda: ra.cross_attention_fwd(q, k, k),
                lambda: ra.ra_cross_fwd(q, k, k, 0.1, q[:, :2], lse, ws), lambda: ra.ra_cross_fwd(q, k, k, 0.1, q, lse[:1], ws),
                lambda: ra.ra_cross_fwd(q, k, k, 0.1, q, lse.double(), ws),
                lambda: ra.cross_attention_bwd(q, k, k, q, lse, q.float()), lambda: ra.cross_attention_bwd(q, k, k, q, lse.transpose(1, 2), q),
                lambda: ra.ra_cross_bwd(q, k, k, q, q, lse, 0.1, q, k, k.float(), ws),
                lambda: ra.ra_cross_bwd(q, k, k, q, q, lse, 0.1, q, k, k[:, :3], ws)):
        with pytest.raises(ra.RAError):
            bad()
    for i in range(3):
        t = k.narrow(i, 0, 1).expand(*k.shape)
        with pytest.raises(ra.RAError, match="expanded"):
            ra.cross_attention_fwd(q, t, t)


def test_binding_refuses_before_the_library(ra):
    q, k = torch.zeros(2, 8, 4, 16), torch.zeros(2, 8, 2, 16)
    f, w = torch.ones(8, dtype=torch.float64), torch.ones(16)
    pos = torch.zeros(8, dtype=torch.int64)
    ws = torch.zeros(8)
    for bad in (lambda: ra.ra_rotary_fwd(q, k[:, :7], f, q, k), lambda: ra.ra_rotary_fwd(q, k[..., :8], f, q, k),
                lambda: ra.ra_rotary_fwd(q, k.half(), f, q, k), lambda: ra.ra_rotary_fwd(q[0], k, f, q, k),
                lambda: ra.ra_rotary_fwd(q, k, f, k, k), lambda: ra.ra_rotary_fwd(q, k, f, q, None),
                lambda: ra.ra_rotary_fwd(q, None, f, q, k), lambda: ra.ra_rotary_fwd(q, k, None, q, k),
                lambda: ra.ra_rotary_fwd(q, k, f.float(), q, k), lambda: ra.ra_rotary_fwd(q, k, f[None], q, k),
                lambda: ra.ra_rotary_fwd(q, k, f, q, k, positions=pos.int()),
                lambda: ra.ra_rotary_fwd(q, k, f, q, k, positions=pos[:7]),
                lambda: ra.ra_rotary_fwd(q, k, f, q, k, positions=pos[:, None].expand(8, 2).T[:, ::2]),
                lambda: ra.ra_rotary_fwd(q, k, f, q, k, positions=torch.zeros(2, 16, dtype=torch.int64)[:, ::2]),
                lambda: ra.ra_rotary_fwd(q.transpose(2, 3), k, f, q, k),
                lambda: ra.ra_rotary_fwd(q, k, f, q, k),                               # not on a CUDA device
                lambda: ra.rotary_fwd(q, k, f), lambda: ra.rotary_bwd(q, k, f),
                lambda: ra.norm_rotary_fwd(q, k, w, w, f), lambda: ra.norm_rotary_bwd(q, k, q, k, w, w, f),
                lambda: ra.ra_norm_rotary_fwd(q, k, w[:8], w, f, q, k), lambda: ra.ra_norm_rotary_fwd(q, k, w, w.half(), f, q, k),
                lambda: ra.ra_norm_rotary_fwd(q, k, w, w, f, q.half(), k.half()),
                lambda: ra.ra_norm_rotary_bwd(q, k, q, k, w, w, f, q, k, w[:8], w, ws),
                lambda: ra.ra_norm_rotary_bwd(q, k, q, k, w, w, f, q, k, w.double(), w, ws),
                lambda: ra.ra_norm_rotary_bwd(q, k, q, k[:1], w, w, f, q, k, w, w, ws),
                lambda: ra.grad_norm([]), lambda: ra.grad_clip([], 1.0), lambda: ra.grad_norm([w]),
                lambda: ra.ra_grad_norm([w], w, ws), lambda: ra.ra_grad_clip([w], 1.0, ws[0], ws, outs=[])):
        with pytest.raises(ra.RAError):
            bad()
    for t in (q[:1].expand(2, 8, 4, 16), q[:, :1].expand(2, 8, 4, 16), q[:, :, :1].expand(2, 8, 4, 16)):
        with pytest.raises(ra.RAError, match="expanded"):
            ra.ra_rotary_fwd(t, k, f, q, k)
