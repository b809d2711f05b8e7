"""Chains whose tiles are split over several CTA pairs: the splits leave each other partial sums
in memory, each lane of a warp acquires the flag of one split and then reads the sums of all.
The sums are added in a fixed order, so every repetition gives the same bits, alone and beside
a chain on another stream."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

from tests.test_gpu_newton_schulz import gradient  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1000, 333), (333, 4600), (2600, 400), (8000, 300), (919, 5200)])
def test_split_chains_repeat_bit_for_bit(rows, cols):
    import blockwise_exact_attention_ra_gb300 as ra
    g = gradient(rows, cols, 61, "gauss")
    other = gradient(cols, rows, 62, "gauss")
    want, want2 = ra.newton_schulz(g), ra.newton_schulz(other)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(15):
        a = ra.newton_schulz(g)
        b = ra.newton_schulz(other, stream=stream)
        assert torch.equal(a, want)
        stream.synchronize()
        assert torch.equal(b, want2)
    ra.ra_sync_status()
