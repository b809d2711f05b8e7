"""Tensors that lie between each other without sharing an element: slices of one buffer as inputs and
results of the rotary, norm and cross-attention entry points; and what is refused of real tensors."""
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


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("B,N", [(1, 1), (3, 1), (1, 40), (2, 33)])
def test_slices_of_one_buffer(ra, B, N):
    Hq, Hk, d = 6, 2, 64
    freq = ra.rotary_frequencies(d)
    base = rand((B, N, Hq + 2 * Hk, d), torch.bfloat16, 1)
    want = ra.rotary_fwd(base[:, :, :Hq].contiguous(), base[:, :, Hq:Hq + Hk].contiguous(), freq)

    def check(q, k, qo, ko):
        ra.ra_rotary_fwd(q, k, freq, qo, ko)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])

    x = base.clone()                                           # in place; the values beside them stay
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    check(q, k, q, k)
    assert torch.equal(x[:, :, Hq + Hk:], base[:, :, Hq + Hk:])
    x = base.clone()                                           # k's result where v was
    check(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, :Hq], x[:, :, Hq + Hk:])
    x = torch.zeros(B, 2 * N, Hq + 2 * Hk, d, dtype=torch.bfloat16, device="cuda")
    x[:, ::2] = base                                           # rows between rows
    check(x[:, ::2, :Hq], x[:, ::2, Hq:Hq + Hk], x[:, 1::2, :Hq], x[:, 1::2, Hq:Hq + Hk])
    x = torch.zeros(B, 2 * N, Hq + 2 * Hk, d, dtype=torch.bfloat16, device="cuda")
    x[:, :N] = base                                            # one half of each batch entry after the other
    check(x[:, :N, :Hq], x[:, :N, Hq:Hq + Hk], x[:, N:, :Hq], x[:, N:, Hq:Hq + Hk])
    x = torch.zeros(B, N, Hq + 2 * Hk, 2 * d, dtype=torch.bfloat16, device="cuda")
    x[..., :d] = base                                          # heads between heads
    check(x[:, :, :Hq, :d], x[:, :, Hq:Hq + Hk, :d], x[:, :, :Hq, d:], x[:, :, Hq:Hq + Hk, d:])
    x = base.transpose(1, 2).contiguous().transpose(1, 2)      # heads before rows
    check(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, :Hq], x[:, :, Hq + Hk:])
    flat = torch.zeros(4 * base.numel(), dtype=torch.bfloat16, device="cuda")
    n, m = B * N * Hq * d, B * N * Hk * d                      # packed tensors end to end
    q, k, qo, ko = flat[:n].view(B, N, Hq, d), flat[n:n + m].view(B, N, Hk, d), flat[n + m:2 * n + m].view(B, N, Hq, d), \
        flat[2 * n + m:2 * n + 2 * m].view(B, N, Hk, d)
    q.copy_(base[:, :, :Hq])
    k.copy_(base[:, :, Hq:Hq + Hk])
    check(q, k, qo, ko)
    # gradients of the norm written over those of its results, or over the rows
    w = rand((d,), torch.float32, 2)
    dy = rand((B, N, Hq + 2 * Hk, d), torch.bfloat16, 3)
    q, k = base[:, :, :Hq].contiguous(), base[:, :, Hq:Hq + Hk].contiguous()
    ref = ra.norm_rotary_bwd(q, k, dy[:, :, :Hq], dy[:, :, Hq:Hq + Hk], w, w, freq)
    dw = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(ra.ra_norm_rotary_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    over = dy.clone()
    for x in ((over[:, :, :Hq], over[:, :, Hq:Hq + Hk]), (q, k)):
        ra.ra_norm_rotary_bwd(q, k, dy[:, :, :Hq] if x[0] is q else x[0], dy[:, :, Hq:Hq + Hk] if x[0] is q else x[1], w, w, freq,
                              *x, *dw, ws)
        assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1]) and torch.equal(dw[0], ref[2])
    ra.ra_sync_status()


def test_refused(ra):
    x = rand((2, 16, 8, 64), torch.bfloat16, 4)
    q, k = x[:, :8, :4], x[:, 8:, :2]
    freq = ra.rotary_frequencies(64)
    before = x.clone()
    for qo, ko in ((q[:, :, :], x[:, :8, 2:4]), (x[:, 1:9, :4], torch.empty_like(k)), (x[:, :8, 1:5], torch.empty_like(k)),
                   (torch.empty_like(q), x[:, 7:15, :2]), (x.view(2, 32, 4, 64)[:, :8], torch.empty_like(k))):
        with pytest.raises(ra.RAError, match="overlaps"):
            ra.ra_rotary_fwd(q, k, freq, qo, ko)
    c = x[:, :, :4].contiguous()
    lse = torch.empty(2, 4, 16, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    with pytest.raises(ra.RAError, match="overlaps"):
        ra.ra_cross_fwd(c, c, x[:, :, 4:].contiguous(), 0.1, c, lse, ws)
    assert torch.equal(x, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Nq", [1, 200])
def test_cross_slices(ra, dtype, Nq):
    """k and v, and dk and dv, as slices of one buffer; dq written over q, dO or v."""
    B, Nkv, H, d = 2, 150, 2, 64
    kv, q, do = rand((B, Nkv, 2, H, d), dtype, 5), rand((B, Nq, H, d), dtype, 6), rand((B, Nq, H, d), dtype, 7)
    k, v = kv[:, :, 0], kv[:, :, 1]
    o, lse = ra.cross_attention_fwd(q, k, v)
    want = ra.cross_attention_bwd(q, k, v, o, lse, do, grad_dtype=dtype)
    grads = torch.empty_like(kv)
    for over in (None, "q", "do"):
        q2, do2 = q.clone(), do.clone()
        dq = {None: torch.empty_like(q), "q": q2, "do": do2}[over]
        ws = torch.empty(ra.ra_cross_bwd_workspace_bytes(ra._dt(q), ra._cross_shape(q, k, v, None)), dtype=torch.uint8, device="cuda")
        ra.ra_cross_bwd(q2, k, v, o, do2, lse, d ** -0.5, dq, grads[:, :, 0], grads[:, :, 1], ws)
        assert torch.equal(grads[:, :, 0], want[1]) and torch.equal(grads[:, :, 1], want[2])
        assert (dq - want[0]).abs().max() <= 2 * torch.finfo(dtype).eps * want[0].abs().max()
    ra.ra_sync_status()
