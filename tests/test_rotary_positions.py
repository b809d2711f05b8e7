"""CPU-only: positions are given, or follow from an offset, not both."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_exact_attention_ra_gb300 as ra
    return ra


def test_an_offset_does_not_combine_with_positions(ra):
    sh = ra.RaShape(2, 8, 8, 4, 2, 64)
    q, k, qo, ko, more = (ctypes.c_void_p(i << 20) for i in (1, 2, 3, 4, 5))
    for off in (1, -7, 1 << 40):
        rot = ra.RaRotary(64, 4096, 4096, 0, off, 1, 1.0)
        codes = (ra.lib.ra_rotary_fwd(q, k, ra.RA_BF16, sh, rot, 0, qo, ko, sh, None),
                 ra.lib.ra_rotary_bwd(q, k, ra.RA_BF16, sh, rot, 0, qo, ko, ra.RA_BF16, sh, None),
                 ra.lib.ra_norm_rotary_fwd(q, k, ra.RA_BF16, sh, None, None, 0, 1e-6, rot, 0, qo, ko, sh, None),
                 ra.lib.ra_norm_rotary_bwd(q, k, ra.RA_BF16, sh, q, k, ra.RA_BF16, sh, None, None, 0, 1e-6, rot, 0, qo, ko,
                                           ra.RA_BF16, sh, None, None, more, ctypes.c_size_t(1 << 40), None))
        assert codes == (1, 1, 1, 1) and "pos_off" in ra.ra_last_error()
