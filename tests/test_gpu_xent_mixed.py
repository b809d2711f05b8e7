"""dx and dw of different types from one launch.  An epilogue warp then goes from pieces of
fp32 values, which fill both of its staging buffers, to 16-bit ones, which fill one: a copy
out of a buffer has to be done with it before the next piece is staged there.  What one
gradient holds must not depend on the other's type: each is compared bit for bit with what
calls with one type for both give, over repeated calls."""
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


# T, D, V, block: dx split into fp32 planes beside 16-bit dw, whose tiles of few tokens are two
# k-slabs long; fp32 dw first (more tokens than entries) beside 16-bit dx; several blocks, whose
# dx is summed in fp32
CASES = [(2, 264, 20011, 20011), (4, 264, 20011, 20011), (16, 520, 9000, 9000), (17, 264, 20011, 20011),
         (64, 264, 20011, 20011), (100, 264, 20011, 20011), (128, 520, 10007, 10007), (777, 520, 10007, 10007),
         (5000, 264, 700, 700), (33000, 72, 8400, 4100)]


@pytest.mark.parametrize("T,D,V,block", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients_do_not_depend_on_each_others_type(ra, T, D, V, block, dtype):
    x, w, y, g = make(T, D, V, dtype, T + V)
    _, lse = ra.xent_fwd(x, w, y)

    def grads(dx_dtype, dw_dtype):
        return ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=dx_dtype, dw_dtype=dw_dtype)

    dx, dw = grads(torch.float32, torch.float32)
    dx16, dw16 = grads(dtype, dtype)
    # the 16-bit outputs are the fp32 sums rounded once
    assert torch.equal(dx16, dx.to(dtype)) and torch.equal(dw16, dw.to(dtype))
    for _ in range(20):
        a, b = grads(torch.float32, dtype)
        c, d = grads(dtype, torch.float32)
        assert torch.equal(a, dx) and torch.equal(b, dw16) and torch.equal(c, dx16) and torch.equal(d, dw)
    ra.ra_sync_status()
