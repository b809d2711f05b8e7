"""CPU-only: what the rotary, norm and cross-attention entry points refuse because a result lies over
another tensor.  (Calls that they take are in test_gpu_layer_overlap.py.)"""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_exact_attention_ra_gb300 as ra
    return ra


M = 1 << 20
B, N, HQ, HK, D = 2, 8, 4, 2, 64
Q, K = B * N * HQ * D * 2, B * N * HK * D * 2  # bytes of 16-bit queries and keys


def at(mb, extra=0):
    return ctypes.c_void_p(mb * M + extra)


def shape(ra, **kw):
    d = dict(B=B, N_q=N, N_kv=N, Hq=HQ, Hkv=HK, d=D)
    d.update(kw)
    return ra.RaShape(*[d.get(n, 0) for n, _ in ra.RaShape._fields_])


def refused(ra, code):
    return code == 1 and "overlaps" in ra.ra_last_error()


def test_rotary(ra):
    rot = ra.RaRotary(64, 4096, None, 0, 0, 1, 1.0)
    wide = shape(ra, q_rstride=2 * HQ * D)

    def plain(q=at(1), k=at(2), qo=at(3), ko=at(4), sh=None, osh=None, dt=ra.RA_BF16):
        return ra.lib.ra_rotary_fwd(q, k, dt, sh or shape(ra), rot, 0, qo, ko, osh or shape(ra), None)

    def back(q=at(1), k=at(2), qo=at(3), ko=at(4), sh=None, osh=None, gdt=ra.RA_F32):
        return ra.lib.ra_rotary_bwd(q, k, ra.RA_F32, sh or shape(ra), rot, 0, qo, ko, gdt, osh or shape(ra), None)

    def norm(q=at(1), k=at(2), qo=at(3), ko=at(4), sh=None, osh=None):
        return ra.lib.ra_norm_rotary_fwd(q, k, ra.RA_BF16, sh or shape(ra), None, None, 0, 1e-6, rot, 0, qo, ko, osh or shape(ra),
                                         None)

    def norm_back(q=at(1), k=at(2), qo=at(3), ko=at(4), sh=None, osh=None, dqo=at(5), dko=at(6)):
        return ra.lib.ra_norm_rotary_bwd(q, k, ra.RA_BF16, sh or shape(ra), dqo, dko, ra.RA_BF16, shape(ra), None, None, 0, 1e-6,
                                         rot, 0, qo, ko, ra.RA_BF16, osh or shape(ra), None, None, at(7),
                                         ctypes.c_size_t(1 << 40), None)

    for call in (plain, back, norm, norm_back):
        assert refused(ra, call(qo=at(3), ko=at(3)))                       # the results over each other
        assert refused(ra, call(qo=at(4, -16)))                            # their ends
        assert refused(ra, call(qo=at(2))) and refused(ra, call(ko=at(1)))  # over the other's input
        assert refused(ra, call(qo=at(1, 16)))                             # its own, not in place
        assert refused(ra, call(osh=wide, qo=at(1)))                       # its own at other strides
        assert refused(ra, call(ko=at(1, D * 2)))
    assert refused(ra, back(gdt=ra.RA_BF16, qo=at(1)))                     # another type in place
    assert refused(ra, norm_back(qo=at(6))) and refused(ra, norm_back(qo=at(5, 64))) and refused(ra, norm_back(ko=at(5)))
    # one row of a head of a fused buffer, in an axis that only one of the two has
    fused = dict(q_rstride=(HQ + 2 * HK) * D, kv_rstride=(HQ + 2 * HK) * D)
    both = shape(ra, **fused)
    for head in (0, HQ - 1):
        assert refused(ra, plain(sh=both, osh=both, k=at(1, HQ * D * 2), qo=at(3), ko=at(1, head * D * 2)))
    one = shape(ra, Hkv=1, **fused)
    assert refused(ra, plain(sh=one, osh=one, k=at(1, HQ * D * 2), qo=at(3), ko=at(1, (HQ - 1) * D * 2 + 32)))
    assert refused(ra, plain(sh=one, osh=one, k=at(1, HQ * D * 2), qo=at(3), ko=at(1, 7 * 8 * D * 2)))  # the last row's first head


def test_cross(ra):
    for nq in (1, 300):                                                     # both kernels
        sh = shape(ra, N_q=nq)

        def fwd(q=at(1), k=at(2), v=at(3), o=at(4), odt=ra.RA_BF16, sh=sh):
            return ra.lib.ra_cross_fwd(q, k, v, ra.RA_BF16, sh, None, 0, 0.1, o, odt, at(5), at(6), ctypes.c_size_t(1 << 40), None)

        def bwd(q=at(1), k=at(2), v=at(3), o=at(4), do=at(5), dq=at(7), dk=at(9), dv=at(11), gdt=ra.RA_BF16, sh=sh):
            return ra.lib.ra_cross_bwd(q, k, v, o, ra.RA_BF16, do, at(13), ra.RA_BF16, sh, None, 0, 0.1, dq, dk, dv, gdt,
                                       at(14), ctypes.c_size_t(1 << 40), None)

        for name in "qkv":
            assert refused(ra, fwd(**{name: at(4)})) and refused(ra, fwd(**{name: at(4, 16)}))
        assert refused(ra, fwd(q=at(4), odt=ra.RA_F32))
        for grad in ("dk", "dv"):
            for where in (1, 2, 3, 5):
                assert refused(ra, bwd(**{grad: at(where)}))
            assert refused(ra, bwd(dq=at(9 if grad == "dk" else 11, 16)))
        assert refused(ra, bwd(dv=at(9))) and refused(ra, bwd(dv=at(9, K - 16)))
