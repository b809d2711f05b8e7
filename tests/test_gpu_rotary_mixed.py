"""Gradients in fp32 of 16-bit rows are formed as those of fp32 rows are: the same values in fp32
give the same bits."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 32, False), (80, 20, False), (64, 64, True)])
def test_fp32_gradients_of_rows_in_16_bits(ra, dtype, d, rot, interleaved):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    q, k, dq, dk = (torch.randn((2, 333, h, d), generator=g, device="cuda") for h in (6, 2, 6, 2))
    w = 1 + 0.2 * torch.randn(d, generator=g, device="cuda")
    q, k = q.to(dtype), k.to(dtype)
    freq = ra.rotary_frequencies(rot)
    where = dict(interleaved=interleaved, pos_off=100000, grad_dtype=torch.float32)
    got = ra.norm_rotary_bwd(q, k, dq, dk, w, None, freq, **where)
    want = ra.norm_rotary_bwd(q.float(), k.float(), dq, dk, w, None, freq, **where)
    ra.ra_sync_status()
    for a, b in zip(got, want):
        assert a.dtype == torch.float32 and torch.equal(a, b)
