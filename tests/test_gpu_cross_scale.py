"""Cross attention's gradients for output gradients of any size, against the fp64 oracle.

The gradients are linear in dO, so that the bounds for dO of size 1 hold at every size.  In
2-norm: 2e-3, four times the half step 2^-11 of the fp16 operands P and dS (each is rounded once, dO's
copy times a power of two not at all), and what is left of two fp32 sums where dP and D agree:
delta = 16 x 2^-23 of sum |dO| |v|, which moves a row of dq by at most scale delta max |k| and a row of
dk by scale delta max |q| times its column's sum of P; with R rows of queries the 2-norms are within
sqrt(R) and R of that.  An o in 16 bits enters D only past 4 d keys without `precise`, which these
calls leave out."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests._parity import f64

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


def inputs(B, Nq, Nkv, Hq, Hkv, d, dtype, seed):
    """Queries lean towards a key each; dO of size 1, of few bits (so that it is exact times a power of two)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k, v = (torch.randn((B, Nkv, Hkv, d), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((B, Nq, Hq, d), generator=g, device="cuda")
    pick = torch.randint(0, Nkv, (B, Nq, Hkv), generator=g, device="cuda")
    at = k.gather(1, pick[..., None].expand(B, Nq, Hkv, d))
    q += 0.5 * torch.rand((B, Nq, Hq, 1), generator=g, device="cuda") * at.repeat_interleave(Hq // Hkv, dim=2)
    do = torch.randn((B, Nq, Hq, d), generator=g, device="cuda").to(BF).float()
    return q.to(dtype), k.to(dtype), v.to(dtype), do


def near(name, got, want, left, rel=2e-3):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= rel * norm + left, f"{name}: off by {err / norm:.3g} of its norm, limit {rel + left / norm:.3g}"


def check(ra, q, k, v, do, lens=None, parts=((slice(None), slice(None)),)):
    """Both ways to call; each part (batch entries, key heads) against its own norm."""
    B, Nq, Hq, d = q.shape
    Hkv, scale = k.shape[2], d ** -0.5
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = oracle.cross_attention(f64(q), f64(k), f64(v), scale, lens, f64(do))[2:]
    for precise, o_dtype in ((False, torch.float32), (True, q.dtype)):
        o, lse = ra.cross_attention_fwd(q, k, v, kv_len, o_dtype=o_dtype, precise=precise)
        got = ra.cross_attention_bwd(q, k, v, o, lse, do, kv_len, precise=precise)
        ra.ra_sync_status()
        for b, g in parts:
            qh = range(Hkv)[g] if isinstance(g, slice) else range(g, g + 1)
            qs = slice(qh.start * (Hq // Hkv), qh.stop * (Hq // Hkv))
            gs = slice(qh.start, qh.stop)
            Q, K, V, G = f64(q)[b, :, qs], f64(k)[b, :, gs], f64(v)[b, :, gs], np.abs(f64(do)[b, :, qs])
            delta = scale * 16 * 2.0 ** -23 * G.reshape(-1, d).max(axis=0) @ np.abs(V).reshape(-1, d).max(axis=0)
            R = G.size // d
            near(f"dq {precise}", got[0][b, :, qs], want[0][b, :, qs], R ** 0.5 * delta * np.linalg.norm(K, axis=-1).max())
            near(f"dk {precise}", got[1][b, :, gs], want[1][b, :, gs], R * delta * np.linalg.norm(Q, axis=-1).max())
            near(f"dv {precise}", got[2][b, :, gs], want[2][b, :, gs], 0.0)
    return got, want


@pytest.mark.parametrize("Nkv", [77, 1000, 40000])
@pytest.mark.parametrize("dtype,exponent", [(BF, -90), (BF, -40), (BF, -27), (BF, -14), (BF, 0), (BF, 12), (BF, 80), (HF, -20), (HF, -13),
                                            (HF, 0), (HF, 12)])
def test_any_size(ra, dtype, exponent, Nkv):
    d = 64 if Nkv == 1000 else 128
    q, k, v, do = inputs(1, 140, Nkv, 2, 1, d, dtype, Nkv)
    check(ra, q, k, v, (do * 2.0 ** exponent).to(dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_sequence_in_a_padded_batch(ra, dtype):
    """Batch entries and heads whose gradients differ by 2^20 and more keep their digits each."""
    q, k, v, do = inputs(3, 70, 900, 4, 2, 64, dtype, 5)
    for b, g, e in ((0, 0, 0), (0, 1, -10), (1, 0, -12), (1, 1, 10), (2, 0, 3), (2, 1, -9)):
        do[b, :, 2 * g:2 * g + 2] *= 2.0 ** (2 * e if dtype == BF else e)
    lens = [900, 33, 512]
    for b, n in enumerate(lens):
        k[b, n:] = v[b, n:] = 0
    parts = [(slice(b, b + 1), g) for b in range(3) for g in range(2)]
    check(ra, q, k, v, do.to(dtype), lens, parts)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_small_rows_beside_large_ones(ra, dtype):
    """Rows whose dO is 2^-10 of the others' keep their digits in dq."""
    q, k, v, do = inputs(1, 260, 1000, 2, 2, 64, dtype, 6)
    do[:, 1::2] *= 2.0 ** -10
    got, want = check(ra, q, k, v, do.to(dtype))
    G, V, K = np.abs(f64(do)[:, 1::2]), np.abs(f64(v)), f64(k)
    delta = 0.125 * 16 * 2.0 ** -23 * G.reshape(-1, 64).max(axis=0) @ V.reshape(-1, 64).max(axis=0)
    near("dq of the small rows", got[0][:, 1::2], want[0][:, 1::2], (G.size / 64) ** 0.5 * delta * np.linalg.norm(K, axis=-1).max())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_that_share_two_keys_of_many(ra, dtype):
    """P of 1/2 among 40000 keys, where dS is as large as a quarter of dP's range."""
    q, k, v, do = inputs(1, 150, 40000, 2, 1, 64, dtype, 7)
    k[:, :2] = torch.sign(k[:, :2].float()).to(dtype)
    q.copy_(((k[:, 0] + k[:, 1]).float() * 2.5)[:, None].expand_as(q))      # scores of about 20
    for e in (0, 7, 12):
        check(ra, q, k, v, (do * 2.0 ** e).to(dtype))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_nothing_and_infinities(ra, dtype):
    q, k, v, do = inputs(2, 140, 300, 2, 1, 64, dtype, 8)
    kv_len = torch.tensor([300, 131], dtype=torch.int32, device="cuda")
    k[1, 131:], v[1, 131:] = float("nan"), 6e4                  # not looked at
    o, lse = ra.cross_attention_fwd(q, k, v, kv_len)
    for g in ra.cross_attention_bwd(q, k, v, o, lse, torch.zeros_like(q), kv_len):
        assert not g.any()
    small = (do * 2.0 ** -9).to(dtype)
    small[1] = 0
    clean = ra.cross_attention_bwd(q, k, v, o, lse, small, kv_len)
    assert not any(g[1].any() for g in clean)
    small[0, 3, 1, 5], small[0, 7, 0, 2] = float("inf"), float("nan")
    got = ra.cross_attention_bwd(q, k, v, o, lse, small, kv_len)
    ra.ra_sync_status()
    rows = torch.ones(140, 2, dtype=torch.bool, device="cuda")
    rows[3, 1] = rows[7, 0] = False
    assert not got[0][0][~rows].isfinite().any(dim=-1).any() and torch.isnan(got[1][0]).all()
    a, b = got[0][0][rows].double(), clean[0][0][rows].double()
    assert (a - b).norm() <= 2 * 2e-3 * b.norm()              # another power of two at most
    assert not got[0][1].any() and not got[1][1].any() and not got[2][1].any()
    zero = torch.zeros_like(v)
    o, lse = ra.cross_attention_fwd(q, k, zero, kv_len)
    dq, dk, dv = ra.cross_attention_bwd(q, k, zero, o, lse, (do * 2.0 ** -9).to(dtype), kv_len)
    assert not dq.any() and not dk.any() and dv[0].any() and not dv[1, 131:].any()
    ra.ra_sync_status()


def test_large_bf16_gradients_set_no_status(ra):
    """dO past fp16's range is held times a power of two; v, q and k are copied as they are and report theirs."""
    q, k, v, do = inputs(1, 200, 300, 2, 2, 64, BF, 9)
    check(ra, q, k, v, (do * 2.0 ** 20).to(BF))
    v[0, 5, 0, 1] = 1e5
    o, lse = ra.cross_attention_fwd(q, k, v)
    ra.cross_attention_bwd(q, k, v, o, lse, do.to(BF))
    with pytest.raises(ra.RAError, match="RANGE"):
        ra.ra_sync_status()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("exponent", [-80, -30, 0, 90])
@pytest.mark.parametrize("Nq", [2, 200])
def test_rows_beside_a_lost_one(ra, Nq, exponent, bad):
    """Rows of dO without a finite element leave the others, of any size, their dq.  (Each reader of
    rows meets lost ones before it meets others.)"""
    q, k, v, do = inputs(1, Nq, 300, 2, 1, 64, BF, 10)
    do = do * 2.0 ** exponent
    o, lse = ra.cross_attention_fwd(q, k, v)
    want = oracle.cross_attention(f64(q), f64(k), f64(v), 0.125, None, f64(do))[2]
    lost = do.clone()
    lost[0, :Nq // 2] = bad
    dq, _, _ = ra.cross_attention_bwd(q, k, v, o, lse, lost.to(BF))
    ra.ra_sync_status()
    assert not dq[0, :Nq // 2].isfinite().any()
    G, V = np.abs(f64(do)), np.abs(f64(v))
    delta = 0.125 * 16 * 2.0 ** -23 * G.reshape(-1, 64).max(axis=0) @ V.reshape(-1, 64).max(axis=0)
    near("dq", dq[0, Nq // 2:], want[0, Nq // 2:], Nq ** 0.5 * delta * np.linalg.norm(f64(k), axis=-1).max())
