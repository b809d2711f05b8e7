"""Cross attention of rows whose scores are infinite: a row with a score of +inf or NaN is NaN in o and
lse, a score of -inf counts as a key that is not there (all of them: o = 0, lse = -inf), and other rows
and heads keep their bits.  Sizes: a few queries in one part, in a cluster's, and in parts that a kernel
joins; tiles of queries in one part and several, with P in bf16 terms and with V copied to fp16."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests._parity import f64

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu
SIZES = [(1, 4, 100), (1, 4, 1000), (1, 4, 30000), (64, 3, 500), (1, 150, 700), (1, 150, 9000), (1, 700, 300), (1, 700, 5000)]  # B, Nq, Nkv
INF = float("inf")


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


def inputs(B, Nq, Nkv, dtype):
    """Four query heads, two key heads.  Of the keys column 0 is positive and column 1 of both signs; of the
    queries both are 0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(Nq + Nkv)
    q, k, v, do = (torch.randn(s, generator=g, device="cuda") for s in ((B, Nq, 4, 64), (B, Nkv, 2, 64), (B, Nkv, 2, 64), (B, Nq, 4, 64)))
    k[..., 0] = k[..., 0].abs() + 0.25
    k[:, ::2, :, 1], k[:, 1::2, :, 1] = 1.5, -0.5
    q[..., :2] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype), do.to(dtype)


ROWS = [  # query from the end, head, column, value, what the row becomes
    (1, 0, 0, INF, "nan"), (1, 1, 0, -INF, "empty"), (2, 0, 1, INF, "nan"), (2, 3, 1, -INF, "nan"), (1, 2, 5, float("nan"), "nan")]


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,Nq,Nkv", SIZES)
def test_infinite_queries(ra, B, Nq, Nkv, dtype, precise):
    q, k, v, do = inputs(B, Nq, Nkv, dtype)
    clean, clse = ra.cross_attention_fwd(q, k, v, precise=precise)
    bad = torch.zeros(B, Nq, 4, dtype=torch.bool, device="cuda")
    x = q.clone()
    for n, h, c, value, _ in ROWS:
        x[0, Nq - n, h, c] = value
        bad[0, Nq - n, h] = True
    for kv_len in (None, torch.full((B,), Nkv, dtype=torch.int32, device="cuda")):
        o, lse = ra.cross_attention_fwd(x, k, v, kv_len, precise=precise)
        ra.ra_sync_status()
        for n, h, _, _, kind in ROWS:
            row, l = o[0, Nq - n, h], float(lse[0, h, Nq - n])
            if kind == "nan":
                assert row.isnan().all() and np.isnan(l), (n, h)
            else:
                assert not row.any() and l == -INF, (n, h)
        if kv_len is None:
            assert torch.equal(o[~bad], clean[~bad]) and torch.equal(lse.transpose(1, 2)[~bad], clse.transpose(1, 2)[~bad])
    # gradients of the other rows; those of the keys of a head with such a row are lost
    good = ra.cross_attention_bwd(q, k, v, clean, clse, do, precise=precise)
    dq, dk, dv = ra.cross_attention_bwd(x, k, v, o, lse, do, precise=precise)
    ra.ra_sync_status()
    kept = bad[:, :, :, None].expand_as(dq).logical_not()
    assert (dq[kept] - good[0][kept]).abs().max() <= 1e-5 * good[0].abs().max()
    if B > 1:
        assert torch.equal(dk[1:], good[1][1:]) and torch.equal(dv[1:], good[2][1:])
    assert not dq[0, Nq - 1, 1].any() and dq[0, Nq - 1, 0].isnan().all() and dq[0, Nq - 2, 3].isnan().all()
    assert dk[0].isnan().all() and dv[0].isnan().all()


@pytest.mark.parametrize("B,Nq,Nkv", SIZES)
def test_scores_past_fp32(ra, B, Nq, Nkv):
    """Finite bf16 queries and keys whose products are infinite: -inf at some keys, all of a part's among
    them, leaves the row to the others; +inf makes it NaN."""
    q, k, v, _ = inputs(B, Nq, Nkv, torch.bfloat16)
    k[..., 3], q[..., 3] = 0, 0
    k[:, :2 * Nkv // 3, 0, 3] = 1e30      # key head 0: the first two thirds, whole parts of the keys
    k[:, 5::7, 1, 3] = 1e30               # key head 1: here and there
    clean, clse = ra.cross_attention_fwd(q, k, v)
    x = q.clone()
    x[:, -1, :, 3] = -1e10
    x[:, 0, 1, 3] = x[:, 0, 2, 3] = 1e10
    o, lse = ra.cross_attention_fwd(x, k, v)
    ra.ra_sync_status()
    assert o[:, 0, 1:3].isnan().all() and lse[:, 1:3, 0].isnan().all()
    assert torch.equal(o[:, 1:-1], clean[:, 1:-1]) and torch.equal(o[:, 0, 0], clean[:, 0, 0]) and torch.equal(o[:, 0, 3], clean[:, 0, 3])
    assert torch.equal(lse[:, :, 1:-1], clse[:, :, 1:-1])
    # the last row: the same as if those keys were not there, within the rounding of P (2^-11, 2^-25 a key) and sums
    for h in range(4):
        there = (k[0, :, h // 2, 3] == 0).cpu().numpy()
        want, wlse = oracle.cross_attention(f64(q[:1, -1:, h:h + 1]), f64(k[:1, :, h // 2:h // 2 + 1])[:, there],
                                            f64(v[:1, :, h // 2:h // 2 + 1])[:, there], 0.125)
        top = np.abs(f64(v[:1, :, h // 2])).max()
        assert np.abs(f64(o[:1, -1:, h:h + 1]) - want).max() <= top * (2.0 ** -11 + Nkv * 2.0 ** -25 + 1e-5)
        assert abs(float(lse[0, h, -1]) - float(wlse[0, 0, 0])) <= 1e-5 * (1 + abs(float(wlse[0, 0, 0])))
