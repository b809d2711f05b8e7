"""Cross attention on the GPU against the fp64 oracle.

Tolerances, element by element for the forward pass.  u: half a step of o's type.  Scores are
fp32 sums of d <= 128 exact products in at most 16 steps that may round towards zero, so that an
exponent is off by at most e = scale 16 x 2^-23 max_ij sum |q| |k|, and a probability by e twice over
(its own, and those of the sum) and 2^-21 (two hardware exponentials, 2^-22 each).  P is rounded to fp16
(2^-11; below 2^-14 of the row's largest to a multiple of 2^-24, half of which is 2^-25 for each key),
or carried as two bf16 terms (2^-17) or two fp16 terms (2^-22).  The sums over keys: 2^-23 (8 + N / 16).
The backward pass is held to the stated bounds of the 16-bit kernels and, as a whole, to 2e-3 in 2-norm:
four times the half step 2^-11 of its fp16 operands P and dS.  dS = P (dP - D) is what is left of two
fp32 sums, whose own errors stay where dP and D agree (a single key: dS = 0): delta = 16 x 2^-23 of
sum |dO| |v|, and u sum |dO| |o| where D is formed from an o rounded to 16 bits.  Off by P delta, it moves a row
of dq by at most scale delta max |k|, a row of dk by scale delta max |q| times its column's sum of P; with R rows
of queries the 2-norms are within sqrt(R) and R of that."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests._parity import check, f64

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu
U = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


def rand(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def inputs(B, Nq, Nkv, Hq, Hkv, d, dtype, seed):
    return (rand((B, Nq, Hq, d), dtype, seed), rand((B, Nkv, Hkv, d), dtype, seed + 1),
            rand((B, Nkv, Hkv, d), dtype, seed + 2), rand((B, Nq, Hq, d), dtype, seed + 3))


def length_tensor(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_forward(q, k, v, scale, lens, o, lse, p_error):
    Q, K, V = f64(q), f64(k), f64(v)
    if lens is not None:  # what lies past the lengths may be anything
        for b, n in enumerate(lens):
            n = min(max(n, 0), K.shape[1])
            K[b, n:] = V[b, n:] = 0
    want, wlse = oracle.cross_attention(Q, K, V, scale, lens)
    size, _ = oracle.cross_attention(Q, K, np.abs(V), scale, lens)
    N = K.shape[1]
    e = scale * 16 * 2.0 ** -23 * max(np.abs(Q).max(axis=(0, 1, 2)) @ np.abs(K).max(axis=(0, 1, 2)), 0)
    sums = 2.0 ** -23 * (8 + N / 16)
    lim = U[o.dtype] * np.abs(want) * 1.01 + (p_error + 2 * e + 2.0 ** -21 + sums) * size + \
        (N * 2.0 ** -25 * np.abs(V).max() if p_error == 2.0 ** -11 else 0) + 2.0 ** -25
    got = f64(o)
    assert got.shape == want.shape
    err = np.abs(got - want)
    assert (err <= lim).all(), f"o: worst {np.nanmax(err / lim):.3g} times the limit"
    none = wlse == -np.inf
    gl = f64(lse)
    assert (gl[none] == -np.inf).all() and np.isfinite(gl[~none]).all()
    lerr = np.abs(gl[~none] - wlse[~none])
    assert (lerr <= e + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(wlse[~none])).all(), lerr.max()
    assert (got[np.broadcast_to(none.transpose(0, 2, 1)[..., None], got.shape)] == 0).all()
    return want, wlse


def p_error_of(Nq, Hq, Hkv, dtype, precise=False):
    rows = Nq * (Hq // Hkv)
    if rows <= 32:
        return 2.0 ** -17 if dtype == torch.bfloat16 else 2.0 ** -22
    if precise:
        return 2.0 ** -22
    return 2.0 ** -17 if dtype == torch.bfloat16 and rows <= 512 else 2.0 ** -11


FEW = [  # B, Nq, Nkv, Hq, Hkv, d, lens
    (1, 1, 1, 1, 1, 64, None), (2, 1, 15, 4, 4, 128, [3, 15]), (1, 1, 17, 8, 1, 64, None), (3, 1, 300, 8, 2, 128, [0, 1, 299]),
    (1, 5, 1000, 4, 1, 128, None), (2, 8, 129, 4, 1, 64, [128, 129]), (1, 32, 64, 2, 2, 64, None), (1, 16, 5000, 2, 1, 128, [4097]),
    (1, 1, 70000, 2, 2, 64, None), (4, 3, 2048, 5, 5, 128, [2048, 7, -3, 9999]), (1, 2, 33, 32, 2, 64, [16]), (64, 1, 513, 2, 1, 128, None),
]
TILES = [
    (1, 33, 1, 1, 1, 64, None), (1, 33, 130, 4, 4, 128, None), (2, 128, 128, 2, 1, 64, [128, 1]), (1, 129, 127, 2, 2, 128, [64]),
    (3, 200, 300, 4, 2, 64, [0, 129, 300]), (1, 513, 1000, 2, 2, 128, None), (2, 257, 520, 6, 2, 64, [511, 513]),
    (1, 1000, 77, 3, 3, 128, None), (1, 100, 20000, 2, 1, 64, [19999]), (16, 64, 200, 4, 4, 128, [13 * i for i in range(16)]),
    (1, 2049, 384, 1, 1, 128, [383]), (5, 40, 256, 16, 2, 64, None), (1, 8, 640, 8, 1, 128, None),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", FEW + TILES)
def test_forward(ra, case, dtype):
    B, Nq, Nkv, Hq, Hkv, d, lens = case
    q, k, v, _ = inputs(B, Nq, Nkv, Hq, Hkv, d, dtype, 10)
    if lens is not None:  # the keys past a length hold what must not be looked at
        for b, n in enumerate(lens):
            n = min(max(n, 0), Nkv)
            k[b, n:], v[b, n:] = float("nan"), float("inf")
            if n < Nkv:
                v[b, n] = float("nan")
    scale = 1.3 * d ** -0.5
    for precise in (False, True) if case in TILES[3:6] else (False,):
        for o_dtype in (torch.float32, dtype):
            o, lse = ra.cross_attention_fwd(q, k, v, length_tensor(lens), scale, o_dtype, precise=precise)
            ra.ra_sync_status()
            assert o.dtype == o_dtype
            check_forward(q, k, v, scale, lens, o, lse, p_error_of(Nq, Hq, Hkv, dtype, precise))
    again, _ = ra.cross_attention_fwd(q, k, v, length_tensor(lens), scale, dtype, precise=precise)
    assert torch.equal(o, again)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Nkv,d,lens,precise", [
    (3, 128, None, False), (2, 64, None, False), (128, 128, None, False), (256, 64, None, False), (512, 128, None, False),
    (700, 128, [700, 40, 0, 130], False), (1000, 64, [3, 1000, 256, 257], False), (900, 128, None, True),
    (1500, 128, [9, 1500, 1200, 700], True)])
def test_gradients_from_an_o_in_16_bits(ra, dtype, Nkv, d, lens, precise):
    """o as the forward pass returns it in the inputs' type, rows that lean towards one key each.  In
    the 2-norm, entry by entry: the gradients' own rounding (uniform within half a step of values
    spread over a binade: at most u / sqrt(3), 0.58 u), for bf16 also that of P and dS to one fp16
    term (2.8e-4 each at most), and 2e-5 for the rest.  An o rounded to 16 bits would leave up to three times u
    where few keys share a row; past 4 d keys, without `precise`, it may leave another 0.58 u: |O| is
    at most that of one value, and dP - D that of a difference of two."""
    B, Nq, Hq, Hkv = (2 if lens is None else 4), 300, 4, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(Nkv + d)
    k, v, do = (torch.randn(s, generator=g, device="cuda") for s in ((B, Nkv, Hkv, d), (B, Nkv, Hkv, d), (B, Nq, Hq, d)))
    q = torch.randn((B, Nq, Hq, d), generator=g, device="cuda")
    for b in range(B):
        n = Nkv if lens is None else max(lens[b], 1)
        pick = torch.randint(0, n, (Nq, Hkv), generator=g, device="cuda")
        at = k[b].gather(0, pick[..., None].expand(Nq, Hkv, d))
        q[b] += 0.5 * torch.rand((Nq, Hq, 1), generator=g, device="cuda") * at.repeat_interleave(Hq // Hkv, dim=1)
    q, k, v, do = (t.to(dtype) for t in (q, k, v, do))
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = ra.cross_attention_fwd(q, k, v, kv_len, o_dtype=dtype)
    got = ra.cross_attention_bwd(q, k, v, o, lse, do, kv_len, grad_dtype=dtype, precise=precise)
    ra.ra_sync_status()
    want = oracle.cross_attention(f64(q), f64(k), f64(v), d ** -0.5, lens or [Nkv] * B, f64(do))[2:]
    u = torch.finfo(dtype).eps / 2
    for b in range(B):
        n = Nkv if lens is None else lens[b]
        if n == 0:
            assert not any(t[b].any() for t in got)
            continue
        limit = 0.58 * u + (5.6e-4 if dtype == torch.bfloat16 else 0) + 2e-5
        for name, x, y in zip(("dq", "dk", "dv"), got, want):
            lim = limit + (0.58 * u if n > 4 * d and not precise and name != "dv" else 0)
            err = np.linalg.norm(f64(x)[b] - y[b]) / np.linalg.norm(y[b])
            assert err <= lim, f"{name} of entry {b} ({n} keys): {err:.3g}, limit {lim:.3g}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", TILES + FEW)
def test_backward(ra, case, dtype):
    B, Nq, Nkv, Hq, Hkv, d, lens = case
    if B * Hq * Nq * Nkv * d > 2 ** 30:
        pytest.skip("a long oracle")
    q, k, v, do = inputs(B, Nq, Nkv, Hq, Hkv, d, dtype, 20)
    scale = d ** -0.5
    K, V = f64(k), f64(v)
    if lens is not None:
        for b, n in enumerate(lens):
            n = min(max(n, 0), Nkv)
            K[b, n:] = V[b, n:] = 0
            k[b, n:], v[b, n:] = float("nan"), float("-inf")
    want = oracle.cross_attention(f64(q), K, V, scale, lens, f64(do))
    for precise, grad_dtype, o_dtype in ((False, torch.float32, torch.float32), (True, dtype, dtype)):
        o, lse = ra.cross_attention_fwd(q, k, v, length_tensor(lens), scale, o_dtype, precise=precise)
        grads = ra.cross_attention_bwd(q, k, v, o, lse, do, length_tensor(lens), scale, grad_dtype, precise=precise)
        ra.ra_sync_status()
        for name, got, ref in zip(("dq", "dk", "dv"), grads, want[2:]):
            assert got.dtype == grad_dtype
            # rounding of the result, and of o in the sum dO . O
            off = 0 if grad_dtype == torch.float32 else U[dtype]
            g = f64(got)
            assert np.isfinite(g).all(), name
            err, norm = np.linalg.norm(g - ref), np.linalg.norm(ref)
            delta = scale * (16 * 2.0 ** -23 * (np.abs(f64(do)).max(axis=(0, 1, 2)) @ np.abs(V).max(axis=(0, 1, 2))) +
                             off * (np.abs(f64(do)) * np.abs(want[0])).sum(axis=-1).max())
            R = B * Nq * Hq
            left = {"dq": R ** 0.5 * delta * np.linalg.norm(K, axis=-1).max(),
                    "dk": R * delta * np.linalg.norm(f64(q), axis=-1).max(), "dv": 0.0}[name]
            assert err <= (2e-3 + 2 * off) * norm + left, f"{name} {precise}: {err / max(norm, 1e-30):.3g}"
            if norm and np.abs(ref).max() < 4:
                check(name, g, ref, dtype)
        if lens is not None:
            for b, n in enumerate(lens):
                assert not grads[1][b, max(n, 0):].any() and not grads[2][b, max(n, 0):].any()
        again = ra.cross_attention_bwd(q, k, v, o, lse, do, length_tensor(lens), scale, grad_dtype, precise=precise)
        assert torch.equal(again[1], grads[1]) and torch.equal(again[2], grads[2])


@pytest.mark.parametrize("Nq", [1, 3, 200])
def test_layouts(ra, Nq):
    """Heads before rows, slices of fused projections, rows with space between them; what lies
    between is left as it was."""
    B, Nkv, H, d = 2, 300, 4, 64
    q0, k0, v0, do0 = inputs(B, Nq, Nkv, H, H, d, torch.bfloat16, 30)
    scale = d ** -0.5
    lens = length_tensor([300, 131])
    o0, lse0 = ra.cross_attention_fwd(q0, k0, v0, lens, scale)
    g0 = ra.cross_attention_bwd(q0, k0, v0, o0, lse0, do0, lens, scale)

    def heads_first(t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def spaced(t):
        buf = torch.full((B, t.shape[1], t.shape[2], d + 8), 5.0, dtype=t.dtype, device="cuda")
        buf[..., :d] = t
        return buf[..., :d]

    kv = torch.stack((k0, v0), dim=2)
    for qf, kvf in ((heads_first, lambda i: heads_first((k0, v0)[i])), (spaced, lambda i: kv[:, :, i])):
        q, do, k, v = qf(q0), qf(do0), kvf(0), kvf(1)
        o = qf(torch.zeros_like(q0).float())
        lse = torch.empty_like(lse0)
        shape = ra._cross_shape(q, k, v, lens)
        ws = torch.empty(ra.ra_cross_fwd_workspace_bytes(ra.RA_BF16, shape), dtype=torch.uint8, device="cuda")
        ra.ra_cross_fwd(q, k, v, scale, o, lse, ws, lens)
        assert torch.equal(o, o0) and torch.equal(lse, lse0)
        dq = qf(torch.zeros_like(q0).float())
        dk, dv = ra.empty_like_layout(k, torch.float32), ra.empty_like_layout(k, torch.float32)
        ws = torch.empty(ra.ra_cross_bwd_workspace_bytes(ra.RA_BF16, shape), dtype=torch.uint8, device="cuda")
        ra.ra_cross_bwd(q, k, v, o, do, lse, scale, dq, dk, dv, ws, lens)
        assert torch.equal(dk, g0[1]) and torch.equal(dv, g0[2])
        assert (dq - g0[0]).abs().max() <= 1e-5 * g0[0].abs().max()  # fp32 sums over three tiles in any order
        if qf is spaced:
            assert (o._base[..., d:] == 5).all() and (dq._base[..., d:] == 5).all()
    ra.ra_sync_status()


def test_as_the_ring_without_a_mask(ra):
    """Keys of the queries' own length: what the ring computes without a mask."""
    q, k, v, do = inputs(1, 512, 512, 4, 2, 128, torch.bfloat16, 40)
    o, lse = ra.cross_attention_fwd(q, k, v)
    ro, rl = ra.ring_attention_fwd(q, k, v, 2, False)
    assert (o - ro).abs().max() < 2.0 ** -9 * ro.abs().max() and (lse - rl).abs().max() < 1e-5
    for a, b in zip(ra.cross_attention_bwd(q, k, v, o, lse, do), ra.ring_attention_bwd(q, k, v, ro, rl, do, 2, False)):
        assert (a - b).norm() < 2e-3 * b.norm()


def test_extreme_scores(ra):
    """Rows with one overwhelming key, scores that grow along the keys, and infinities among the queries."""
    for Nq in (2, 150):
        q, k, v, _ = inputs(1, Nq, 700, 2, 2, 64, torch.float16, 50)
        k *= torch.linspace(0.01, 6, 700, device="cuda").to(torch.float16)[None, :, None, None]
        q *= 4
        o, lse = ra.cross_attention_fwd(q, k, v, None, 0.5)
        ra.ra_sync_status()
        want, wlse = oracle.cross_attention(f64(q), f64(k), f64(v), 0.5)
        e = 0.5 * 16 * 2.0 ** -23 * (np.abs(f64(q)).max(axis=(0, 1, 2)) @ np.abs(f64(k)).max(axis=(0, 1, 2)))
        assert np.abs(f64(o) - want).max() <= (2 * e + 2.0 ** -11 + 1e-5) * np.abs(f64(v)).max() + 700 * 2.0 ** -25 * 5
        assert np.abs(f64(lse) - wlse).max() <= e + 1e-5 * np.abs(wlse).max()
        q[0, 1, 0, 0] = float("nan")
        o2, lse2 = ra.cross_attention_fwd(q, k, v, None, 0.5)
        assert o2[0, 1, 0].isnan().all() and torch.equal(o2[0, 0], o[0, 0]) and torch.equal(o2[0, 1, 1], o[0, 1, 1])
        assert lse2[0, 0, 1].isnan() and int(lse2.isnan().sum()) == 1
        do = rand(q.shape, torch.float16, 53)
        dq, dk, dv = ra.cross_attention_bwd(q, k, v, o2, lse2, do, None, 0.5)
        assert dq[0, 1, 0].isnan().all() and not dq[0, 0].isnan().any() and not dq[0, 1, 1].isnan().any()
        assert dk[:, :, 0].isnan().all() and dv[:, :, 0].isnan().all() and not dk[:, :, 1].isnan().any()
    ra.ra_sync_status()


def test_differences(ra):
    """Gradients against differences of the forward pass, along a random direction of each input (fp16
    inputs of few bits and steps that are exact in them; fp32 o).  The difference's own error: h^2 / 6 of a
    third derivative, and o's 2^-11 over h on a sum of 2 x 40 x 64 terms that varies like its root."""
    B, Nq, Nkv, H, d = 1, 40, 70, 2, 64
    q, k, v, do = (torch.round(t.float() * 16).clamp(-48, 48).div(16).to(torch.float16) for t in inputs(B, Nq, Nkv, H, H, d, torch.float16, 60))
    o, lse = ra.cross_attention_fwd(q, k, v, precise=True)
    grads = ra.cross_attention_bwd(q, k, v, o, lse, do, precise=True)
    h = 2.0 ** -5
    for i, name in enumerate("qkv"):
        x = (q, k, v)[i]
        step = torch.sign(rand(x.shape, torch.float32, 61 + i))

        def f(s):
            y = [q, k, v]
            y[i] = (x.float() + s * h * step).to(torch.float16)
            return float((ra.cross_attention_fwd(*y, precise=True)[0].double() * do.double()).sum())

        want = float((grads[i].double() * step.double()).sum())
        size = float(grads[i].double().norm())
        assert abs((f(1) - f(-1)) / (2 * h) - want) < 2e-2 * size + 1e-2 * abs(want), name


def test_rows_far_apart(ra):
    """Offsets past 2^31 elements: a batch stride of that size, and a long cache."""
    B, Nkv, H, d = 2, 300, 1, 64
    big = torch.zeros(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((B, Nkv, H, d), (2 ** 31, d, d, 1))
    v2 = torch.zeros(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    v = v2.as_strided((B, Nkv, H, d), (2 ** 31, d, d, 1))
    k.copy_(rand((B, Nkv, H, d), torch.bfloat16, 70))
    v.copy_(rand((B, Nkv, H, d), torch.bfloat16, 71))
    for Nq in (1, 40):
        q = rand((B, Nq, H, d), torch.bfloat16, 72)
        o, lse = ra.cross_attention_fwd(q, k, v)
        p, pl = ra.cross_attention_fwd(q, k.contiguous(), v.contiguous())
        assert torch.equal(o, p) and torch.equal(lse, pl)
    del big, v2, k, v
    N = 2 ** 24 + 77                                    # 2^31 + elements of keys of two heads of 64
    k = torch.zeros(1, N, 2, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[0, -1] = 4.0                                      # score 4 * 64 * scale = 32 against 0
    v[0, -1] = 2.0
    o, lse = ra.cross_attention_fwd(q, k, v)
    p = 1 / (1 + (N - 1) * np.exp(-32.0))
    assert (o - 2 * p).abs().max() < 1e-4 and (lse - (32 - np.log(p))).abs().max() < 1e-4
    ra.ra_sync_status()


@pytest.mark.parametrize("Nq", [1, 300])
def test_streams_graphs_and_refusals(ra, Nq):
    q, k, v, do = inputs(2, Nq, 700, 4, 2, 64, torch.bfloat16, 80)
    lens = length_tensor([700, 300])
    want = ra.cross_attention_fwd(q, k, v, lens)
    grads = ra.cross_attention_bwd(q, k, v, *want, do, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ra.cross_attention_fwd(q, k, v, lens, stream=side)
    g2 = ra.cross_attention_bwd(q, k, v, *got, do, lens, stream=side)
    side.synchronize()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"] if "address" in b}
    for t in (*got, *g2):
        assert owner[t.data_ptr()] == side.cuda_stream
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(g2[1], grads[1]) and torch.equal(g2[2], grads[2])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = ra.cross_attention_fwd(q, k, v, lens)
            out = ra.cross_attention_bwd(q, k, v, o, lse, do, lens)
        graphs.append((g, o, lse, *out))
    lens.copy_(torch.tensor([17, 0], dtype=torch.int32))  # lengths are read when the graph runs
    q.copy_(rand(q.shape, torch.bfloat16, 81))
    o, lse = ra.cross_attention_fwd(q, k, v, lens)
    out = ra.cross_attention_bwd(q, k, v, o, lse, do, lens)
    for g, *_ in graphs * 2:
        g.replay()
    for _, go, gl, gq, gk, gv in graphs:
        assert torch.equal(go, o) and torch.equal(gl, lse) and torch.equal(gk, out[1]) and torch.equal(gv, out[2])
        assert (gq - out[0]).abs().max() <= 1e-5 * out[0].abs().max()
    with pytest.raises(ra.RAError):
        ra.cross_attention_fwd(q, k.cpu(), v.cpu())
    with pytest.raises(ra.RAError):
        ra.cross_attention_fwd(q, k, v, lens.cpu())
    with pytest.raises(ra.RAError):
        ra.cross_attention_fwd(q.float(), k.float(), v.float())
    ra.ra_sync_status()
