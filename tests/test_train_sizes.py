"""Sizes that do not fit the library's integers are refused, not cut to their low 32 bits (the
library would work on part of the tensor and leave the rest).  Tensors without storage stand for
the large ones; the sizes are checked before the device."""
import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_exact_attention_ra_gb300 as ra
    return ra


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused(ra):
    big = 2 ** 32 + 8
    y, f = meta(4, dtype=torch.int64), meta(4, dtype=torch.float32)
    x, w = meta(4, 16), meta(big, 16)
    for bad in (lambda: ra.xent_fwd(x, w, y), lambda: ra.xent_bwd(x, w, y, f, f),
                lambda: ra.ra_xent_fwd(x, w, y, f, f, f),
                lambda: ra.ra_xent_bwd(x, w, y, f, f, 8, x, w, f),
                lambda: ra.xent_fwd(meta(4, big), meta(9, big), y),
                lambda: ra.newton_schulz(meta(big, 1)), lambda: ra.newton_schulz(meta(1, big)),
                lambda: ra.newton_schulz(meta(big, 1, 1)),
                lambda: ra.ra_newton_schulz(meta(big, 1), meta(big, 1), f)):
        with pytest.raises(ra.RAError, match="2147483647"):
            bad()
    assert ra.ra_xent_fwd_workspace_bytes(ra.RA_BF16, 4, 16, big) == 0
    assert ra.ra_xent_bwd_workspace_bytes(ra.RA_BF16, ra.RA_BF16, 4, 16, big, 8) == 0
    assert ra.ra_newton_schulz_workspace_bytes(1, big, 1) == 0


def test_a_block_past_32_bits_is_the_whole_vocabulary(ra):
    size = ra.ra_xent_bwd_workspace_bytes
    assert size(ra.RA_BF16, ra.RA_BF16, 100000, 64, 3001, 2 ** 32 + 8) == size(ra.RA_BF16, ra.RA_BF16, 100000, 64, 3001, 3001)
    assert size(ra.RA_BF16, ra.RA_BF16, 100000, 64, 3001, 2 ** 31) == size(ra.RA_BF16, ra.RA_BF16, 100000, 64, 3001, 3001)
