"""fp16 gradients of the logits are brought into range by a power of two from max |dloss|.
It follows the loss's scale over the whole range of fp32, so that a power of two in dloss
changes nothing but the exponents of dx and dw."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

from tests.test_gpu_xent import make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


# a product may be split into up to 38 planes; results (and planes) that fall below 2^-126 are
# rounded to a multiple of 2^-149, half a step each
@pytest.mark.parametrize("T", [1, 9, 40, 100])
@pytest.mark.parametrize("k", [-100, -60, 60, 115])
def test_powers_of_two_of_the_loss_gradient(ra, T, k):
    x, w, y, g = make(T, 64, 400, torch.float16, 12, ignored=0.0)
    _, lse = ra.xent_fwd(x, w, y)
    for a, b in zip(ra.xent_bwd(x, w, y, lse, g), ra.xent_bwd(x, w, y, lse, g * 2.0 ** k)):
        assert torch.isfinite(b).all()
        off = (a.double() - b.double() * 2.0 ** -k).abs().max()
        assert float(off) <= 39 * 2.0 ** -150 * 2.0 ** -k
    ra.ra_sync_status()


@pytest.mark.parametrize("T", [9, 40, 100])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_one_unusable_loss_gradient_leaves_the_other_tokens(ra, T, bad):
    # small gradients beside it: without their power of two they would be fp16 subnormals
    x, w, y, g = make(T, 64, 400, torch.float16, 19, ignored=0.0)
    g *= 2.0 ** -30
    g[4] = 0.0
    _, lse = ra.xent_fwd(x, w, y)
    want, _ = ra.xent_bwd(x, w, y, lse, g)
    g[4] = bad
    dx, _ = ra.xent_bwd(x, w, y, lse, g)
    ra.ra_sync_status()
    others = torch.arange(T, device="cuda") != 4
    assert torch.equal(dx[others], want[others]) and not torch.isfinite(dx[4]).any()
