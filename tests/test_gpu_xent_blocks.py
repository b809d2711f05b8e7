"""The backward in several blocks of the vocabulary.  Blocks whose gradient takes less than
256 MB are widened, so each case here has a block past that; the launches are counted to see that
there are as many blocks as the sizes say."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

from tests.test_gpu_xent import check_on_gpu, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


# T, D, V, block.  Launches: each block's logits' gradient, its products, and the sum of its dw's
# planes where the tokens are split (MANY: 17 tiles of dw on 76 pairs); beside them the sum of dx's
# planes where the entries are split (FEW, ODD: one tile of dx), and the scale in fp16
FEW = (40, 8, 6805000, 3400000)      # two terms of the gradient; a last block of 5000
ODD = (17, 16, 17000007, 8000001)    # blocks that begin and end inside tiles; a last block of 1000005
MANY = (33000, 72, 8400, 4100)       # fp32 sums of dx over blocks; a last block of 200


def launches(ra, call):
    before = ra.ra_launch_count()
    out = call()
    return out, ra.ra_launch_count() - before


@pytest.mark.parametrize("case,each,extra", [(FEW, 2, 1), (ODD, 2, 1), (MANY, 3, 0)])
@pytest.mark.parametrize("dtype,dx_dtype,dw_dtype", [(torch.bfloat16, torch.bfloat16, torch.float32),
                                                     (torch.float16, torch.float32, torch.float16)])
def test_blocks_with_gradients_of_two_types(ra, case, each, extra, dtype, dx_dtype, dw_dtype):
    T, D, V, block = case
    assert 2 * T * block > 256 << 20
    x, w, y, g = make(T, D, V, dtype, T)
    y[0], y[1], y[2], y[3] = block - 1, block, 2 * block, V - 1     # on both sides of the blocks' edges
    loss, lse = ra.xent_fwd(x, w, y)
    (dx, dw), n = launches(ra, lambda: ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=dx_dtype, dw_dtype=dw_dtype))
    assert n == each * 3 + extra + (dtype == torch.float16)
    ra.ra_sync_status()
    check_on_gpu(x, w, y, g, loss, lse, dx, dw)


@pytest.mark.parametrize("case", [FEW, MANY])
def test_blocks_keep_inside_their_buffers(ra, case):
    T, D, V, block = case
    guard = 4096
    x, w, y, g = make(T, D, V, torch.bfloat16, 2)
    loss, lse = ra.xent_fwd(x, w, y)
    want = ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16)
    bufs = [torch.full((n + 2 * guard,), 7.0, dtype=torch.bfloat16, device="cuda") for n in (T * D, V * D)]
    dx, dw = (b[guard:-guard].view(-1, D) for b in bufs)
    n = ra.ra_xent_bwd_workspace_bytes(ra.RA_BF16, ra.RA_BF16, T, D, V, block)
    ws = torch.full((n + guard,), 9, dtype=torch.uint8, device="cuda")
    ra.ra_xent_bwd(x, w, y, lse, g, block, dx, dw, ws[:n])
    ra.ra_sync_status()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    for b in bufs:
        assert (b[:guard] == 7).all() and (b[-guard:] == 7).all()
    assert (ws[n:] == 9).all()


@pytest.mark.parametrize("case", [FEW, MANY])
def test_blocks_in_a_graph_and_on_two_streams(ra, case):
    T, D, V, block = case
    first, second = make(T, D, V, torch.float16, 3), make(T, D, V, torch.float16, 4)

    def step(x, w, y, g, stream=None):
        loss, lse = ra.xent_fwd(x, w, y, stream=stream)
        return (loss, lse) + ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=torch.float16, stream=stream)

    want = [step(*first), step(*second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(*a, stream=s) for a, s in zip((first, second), streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    held = [t.clone() for t in first]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = step(*held, stream=streams[0])
    for i, src in enumerate((second, first)):
        for h, s in zip(held, src):
            h.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[1 - i]))
    ra.ra_sync_status()


def test_logits_of_ten_thousand(ra):
    # exponentials of differences alone: nothing overflows, and the gradients stay within the bounds
    x, w, y, g = make(150, 64, 500, torch.bfloat16, 9, scale=1500.0)
    assert float((x.float() @ w.float().T).abs().max()) > 1e4
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g)
    ra.ra_sync_status()
    check_on_gpu(x, w, y, g, loss, lse, dx, dw)
