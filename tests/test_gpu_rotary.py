"""Rotary positions and norms of heads on the GPU against the fp64 oracle, element by element.

Tolerances.  u is half a step of the result's type.  A turned column is x C + x' S in fp32:
C and S carry the sine's and cosine's error (hardware functions within an eighth of a turn, for
16-bit rows: 3.6e-7 and 4.2e-7, and 1e-7 of their argument; else 1.2e-7 of sincospi) and the
product with the amplitude (2^-24), the two products and the sum 2^-24 each: together less than
1e-6 (|x| + |x'|) A for 16-bit rows, 5e-7 for fp32.  The norm's factor r carries a sum of d <= 256
squares in at most 8 + 5 steps (13 x 2^-24, halved by the root), the reciprocal root (2 ulp), and
the product with the weight: 8e-7.  Results below fp16's normal range are off by half its smallest
step, 2^-25."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests._parity import f64

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
    return (torch.randn(shape, generator=g, device="cuda") * 2).to(dtype)


def near(name, got, want, size, u, rel):
    """|got - want| <= u |want| + rel size + 2^-25, element by element."""
    got = f64(got)
    assert got.shape == want.shape, name
    err, lim = np.abs(got - want), u * np.abs(want) * 1.001 + rel * size + 2.0 ** -25
    bad = ~(err <= lim)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / lim):.3g} times the limit"


def turned_size(x, freq, interleaved, amplitude):
    """(|x| + |x'|) amplitude of each column: what a turned one is made of."""
    n, x = len(freq), np.abs(x)
    out = x.copy()
    if interleaved:
        s = x[..., 0:2 * n:2] + x[..., 1:2 * n:2]
        out[..., 0:2 * n:2] = out[..., 1:2 * n:2] = s * amplitude
    else:
        s = x[..., :n] + x[..., n:2 * n]
        out[..., :n] = out[..., n:2 * n] = s * amplitude
    return out


def frequencies(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))


CASES = [  # B, N, Hq, Hkv, d, rot
    (1, 1, 1, 1, 64, 64), (2, 3, 4, 2, 128, 128), (1, 65, 3, 1, 80, 20), (3, 7, 8, 8, 96, 32), (1, 33, 2, 2, 256, 256),
    (2, 5, 6, 3, 128, 34), (1, 130, 2, 1, 32, 2), (2, 9, 5, 5, 8, 8), (1, 17, 4, 4, 64, 0), (1, 11, 2, 1, 40, 38),
    (64, 1, 32, 8, 128, 64), (1, 700, 1, 1, 256, 130), (1, 3000, 2, 2, 16, 16), (1, 19, 2, 2, 248, 240),
]


def kinds(case, dtype):
    """Which of positions, layout and scaling a case takes."""
    i = CASES.index(case) + (torch.float32, torch.bfloat16, torch.float16).index(dtype)
    return ("rows", "given", "far", "batch")[i % 4], bool(i & 1), (1.0, 1.2)[i // 2 % 2]


def positions_of(kind, B, N, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if kind == "rows":
        return None, oracle.rows_to_positions(N, pos_off=11), 11
    if kind == "given":
        p = torch.randint(0, 4096, (N,), generator=g, device="cuda")
    elif kind == "far":
        p = torch.randint(-2 ** 31, 2 ** 31, (B, N), generator=g, device="cuda")
    else:
        p = torch.randint(0, 2 ** 20, (B, N + 3), generator=g, device="cuda")[:, 2:-1]
    return p, p.cpu().numpy(), 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_rotary_and_its_gradient(ra, case, dtype):
    B, N, Hq, Hkv, d, rot = case
    kind, interleaved, amplitude = kinds(case, dtype)
    q, k = rand((B, N, Hq, d), dtype, 1), rand((B, N, Hkv, d), dtype, 2)
    freq = frequencies(rot)
    pos, p, off = positions_of(kind, B, N, 3)
    where = dict(positions=pos, pos_off=off, interleaved=interleaved, amplitude=amplitude)
    rel = 5e-7 if dtype == torch.float32 else 1e-6
    for back in (False, True):
        got = (ra.rotary_bwd if back else ra.rotary_fwd)(q, k, freq, **where)
        ra.ra_sync_status()
        for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
            assert y.dtype == dtype and y.is_contiguous()
            want = oracle.rotary(f64(x), p, freq.cpu().numpy(), interleaved, amplitude, transpose=back)
            size = turned_size(f64(x), freq, interleaved, amplitude)
            near(f"{name} back={back}", y, want, size, U[dtype], rel)
            assert torch.equal(y[..., rot:], x[..., rot:])
        alone, nothing = (ra.rotary_bwd if back else ra.rotary_fwd)(q, None, freq, **where)
        assert nothing is None and torch.equal(alone, got[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_norm_rotary_and_its_gradients(ra, case, dtype):
    B, N, Hq, Hkv, d, rot = case
    kind, interleaved, amplitude = kinds(case, dtype)
    freq = frequencies(rot) if rot else None
    fnp = np.zeros(0) if freq is None else freq.cpu().numpy()
    pos, p, off = positions_of(kind, B, N, 4)
    x = rand((B, N, Hq, d), dtype, 5), rand((B, N, Hkv, d), dtype, 6)
    w = (1 + 0.3 * rand((d,), torch.float32, 7)).to(dtype), (1 + 0.3 * rand((d,), torch.float32, 8)).to(dtype)
    if CASES.index(case) % 5 == 1:
        w = None, w[1]
    eps = 1e-3
    where = dict(positions=pos, pos_off=off, interleaved=interleaved, amplitude=amplitude, eps=eps)
    rel = 2e-6
    y = ra.norm_rotary_fwd(*x, *w, freq, **where)
    eps = float(np.float32(eps))
    for name, a, b, wt in zip("qk", x, y, w):
        n, _ = oracle.head_norm(f64(a), None if wt is None else f64(wt), eps)
        near(name, b, oracle.rotary(n, p, fnp, interleaved, amplitude), turned_size(n, fnp, interleaved, amplitude),
             U[dtype], rel)
    for g_dtype in {dtype, torch.float32}:
        for out_dtype in {dtype, torch.float32}:
            dy = rand((B, N, Hq, d), g_dtype, 9), rand((B, N, Hkv, d), g_dtype, 10)
            got = ra.norm_rotary_bwd(*x, *dy, *w, freq, grad_dtype=out_dtype, **where)
            ra.ra_sync_status()
            for i, name in enumerate("qk"):
                a, wt = f64(x[i]), None if w[i] is None else f64(w[i])
                g = oracle.rotary(f64(dy[i]), p, fnp, interleaved, amplitude, transpose=True)
                dx, dw = oracle.head_norm_bwd(a, g, wt, eps)
                n, r = oracle.head_norm(a, None, eps)
                aw = 1.0 if wt is None else np.abs(wt)
                gs = turned_size(f64(dy[i]), fnp, interleaved, amplitude)
                # g 1e-6, the mean over a row 16 more roundings, r, the products: under 4e-6 of the terms
                size = r * (gs * aw + np.abs(n) * (gs * aw * np.abs(n)).mean(axis=-1, keepdims=True))
                assert got[i].dtype == out_dtype
                near(f"d{name} {g_dtype} {out_dtype}", got[i], dx, size, U[out_dtype], 4e-6)
                # sums over rows: at most 64 in a lane here, 40 more in lanes, warps and blocks, and each term's 4e-6
                total = (gs * np.abs(n)).sum(axis=(0, 1, 2))
                near(f"d{name} weight", got[2 + i], dw, total, U[torch.float32], 4e-6 + 104 * 2.0 ** -24)
            again = ra.norm_rotary_bwd(*x, *dy, *w, freq, grad_dtype=out_dtype, **where)
            assert all(torch.equal(s, t) for s, t in zip(got, again))


@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 24, False), (64, 40, True)])
def test_strides_in_place_and_striped(ra, d, rot, interleaved):
    """Slices of a fused projection, heads before rows, in place, and the ring's striped rows."""
    B, N, H, P = 2, 24, 3, 4
    fused = rand((B, N, 3, H, d), torch.bfloat16, 11)
    q, k = fused[:, :, 0], fused[:, :, 1]
    freq = frequencies(rot)
    where = dict(interleaved=interleaved, P=P, striped=True, pos_off=5)
    want = ra.rotary_fwd(q.contiguous(), k.contiguous(), freq,
                         positions=torch.tensor(oracle.rows_to_positions(N, P, True, 5), device="cuda"), interleaved=interleaved)
    got = ra.rotary_fwd(q, k, freq, **where)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    near("q", got[0], oracle.rotary(f64(q), oracle.rows_to_positions(N, P, True, 5), freq.cpu().numpy(), interleaved),
         turned_size(f64(q), freq, interleaved, 1.0), U[torch.bfloat16], 1e-6)
    heads = torch.zeros(B, H, N, d, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    rows = torch.zeros(B, N, H, d + 8, device="cuda", dtype=torch.bfloat16)
    ra.ra_rotary_fwd(q, k, freq, heads, rows[..., :d], **where)
    assert torch.equal(heads, want[0]) and torch.equal(rows[..., :d], want[1]) and not rows[..., d:].any()
    v = fused[:, :, 2].clone()
    w = rand((d,), torch.float32, 12)
    normed = ra.norm_rotary_fwd(q, k, w, None, freq, **where)
    dy = rand((B, N, H, d), torch.float32, 13), rand((B, N, H, d), torch.float32, 14)
    dx = ra.norm_rotary_bwd(q, k, *dy, w, None, freq, grad_dtype=torch.float32, **where)
    # the gradients in place of their inputs
    g = dy[0].clone(), dy[1].clone()
    dw = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(ra.ra_norm_rotary_bwd_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    ra.ra_norm_rotary_bwd(q, k, *g, w, None, freq, *g, *dw, ws, **where)
    assert all(torch.equal(s, t) for s, t in zip((*g, *dw), dx))
    ra.ra_norm_rotary_bwd(q, None, dy[0], None, w, None, freq, g[0], None, dw[1], None, ws, **where)
    assert torch.equal(g[0], dx[0]) and torch.equal(dw[1], dx[2])
    # the rows in place, the values beside them untouched
    ra.ra_norm_rotary_fwd(q, k, w, None, freq, q, k, **where)
    assert torch.equal(q, normed[0]) and torch.equal(k, normed[1]) and torch.equal(fused[:, :, 2], v)
    # fp32 gradients of the attention to 16-bit ones, as one rounding of the fp32 result
    a = ra.rotary_bwd(dy[0], dy[1], freq, **where)
    b = ra.rotary_bwd(dy[0], dy[1], freq, grad_dtype=torch.float32, **where)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    size = turned_size(f64(dy[0]), freq, interleaved, 1.0)
    for t in (torch.bfloat16, torch.float16):
        c = ra.rotary_bwd(dy[0], dy[1], freq, grad_dtype=t, **where)
        near(str(t), c[0], f64(a[0]), size, U[t], 2e-6)
    ra.ra_sync_status()


def test_rows_of_any_size(ra):
    """Rows of zeros, and values whose squares leave fp32's range; an infinity or a NaN stays in its
    row, and in its pair where nothing norms the row."""
    d = 64
    freq = frequencies(16)
    x = rand((1, 6, 1, d), torch.float32, 15)
    x[0, 0] = 0
    x[0, 1] *= 1e30
    x[0, 2] *= 1e-30
    x[0, 3, 0, 5] = 3e38
    x[0, 4, 0, 40] = float("inf")
    x[0, 5, 0, 3] = float("nan")
    w = rand((d,), torch.float32, 16)
    y, _ = ra.norm_rotary_fwd(x, None, w, None, freq, eps=1e-6)
    n, _ = oracle.head_norm(f64(x[:, :4]), f64(w), float(np.float32(1e-6)))
    near("rows", y[:, :4], oracle.rotary(n, np.arange(4), freq.cpu().numpy()),
         turned_size(n, freq, False, 1.0), U[torch.float32], 2e-6)
    assert not y[0, 0].any()
    assert y[0, 4, 0, 40].isnan() and (y[0, 4, 0, :40] == 0).all() and y[0, 5].isnan().all()
    dy = rand((1, 6, 1, d), torch.float32, 17)
    dx, _, dw, _ = ra.norm_rotary_bwd(x[:, :4], None, dy[:, :4], None, w, None, freq, eps=1e-6)
    g = oracle.rotary(f64(dy[:, :4]), np.arange(4), freq.cpu().numpy(), transpose=True)
    want, want_w = oracle.head_norm_bwd(f64(x[:, :4]), g, f64(w), float(np.float32(1e-6)))
    n, r = oracle.head_norm(f64(x[:, :4]), None, float(np.float32(1e-6)))
    gs = turned_size(f64(dy[:, :4]), freq, False, 1.0)
    size = r * (gs * np.abs(f64(w)) + np.abs(n) * (gs * np.abs(f64(w)) * np.abs(n)).mean(axis=-1, keepdims=True))
    near("dx", dx, want, size, U[torch.float32], 4e-6)
    near("dw", dw, want_w, (gs * np.abs(n)).sum(axis=(0, 1, 2)), U[torch.float32], 1e-5)
    z, _ = ra.rotary_fwd(x, None, freq)
    plain = torch.ones(d, dtype=torch.bool, device="cuda")
    plain[[3, 11]] = False
    assert torch.isfinite(z[0, 4, 0, :40]).all() and z[0, 4, 0, 40] == float("inf")
    assert z[0, 5, 0, [3, 11]].isnan().all() and not z[0, 5, 0, plain].isnan().any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("eps", [0.0, 1e-36])
def test_small_rows_without_eps(ra, dtype, eps):
    """Rows whose squares vanish in fp32, with an eps that does not hide it, beside ordinary ones and
    rows of zeros (0 with an eps, 0 / 0 without)."""
    d, N = 64, 9
    freq = frequencies(64)
    x = rand((1, N, 2, d), dtype, 30)
    small = 1e-5 if dtype == torch.float16 else 1e-25
    x[0, 1::2] *= small
    x[0, 3, 0] *= 0.125
    x[0, 8, 1] = 0
    w = rand((d,), torch.float32, 31)
    y, _ = ra.norm_rotary_fwd(x, None, w, None, freq, eps=eps)
    eps = float(np.float32(eps))
    n, _ = oracle.head_norm(f64(x), f64(w), max(eps, 1e-300))
    rows = N if eps else 8
    near("rows", y[:, :rows], oracle.rotary(n, np.arange(N), freq.cpu().numpy())[:, :rows],
         turned_size(n, freq, False, 1.0)[:, :rows], U[dtype], 2e-6)
    assert eps or (y[0, 8, 1].isnan().all() and not y[0, 8, 0].isnan().any())
    x, dy = x[:, :8].contiguous(), rand((1, 8, 2, d), dtype, 32)
    dx, _, dw, _ = ra.norm_rotary_bwd(x, None, dy, None, w, None, freq, eps=eps, grad_dtype=torch.float32)
    g = oracle.rotary(f64(dy), np.arange(8), freq.cpu().numpy(), transpose=True)
    want, want_w = oracle.head_norm_bwd(f64(x), g, f64(w), eps)
    n, r = oracle.head_norm(f64(x), None, eps)
    gs = turned_size(f64(dy), freq, False, 1.0)
    size = r * (gs * np.abs(f64(w)) + np.abs(n) * (gs * np.abs(f64(w)) * np.abs(n)).mean(axis=-1, keepdims=True))
    near("dx", dx, want, size, U[torch.float32], 4e-6)
    near("dw", dw, want_w, (gs * np.abs(n)).sum(axis=(0, 1, 2)), U[torch.float32], 1e-5)


@pytest.mark.parametrize("rot,interleaved", [(64, False), (20, False), (64, True)])
def test_differences(ra, rot, interleaved):
    """The gradients against differences of the forward pass (fp32; central, step h: h^2 / 6 of third
    derivatives below 10, and 2^-22 of sums near 1 over h, in a sum of 64 such terms)."""
    B, N, H, d = 1, 2, 1, 64
    freq = frequencies(rot)
    x, dy = rand((B, N, H, d), torch.float32, 18) , rand((B, N, H, d), torch.float32, 19)
    w = 1 + 0.3 * rand((d,), torch.float32, 20)

    def f(x, w):
        y, _ = ra.norm_rotary_fwd(x, None, w, None, freq, eps=1e-2, interleaved=interleaved, pos_off=1000)
        return float((y.double() * dy.double()).sum())

    dx, _, dw, _ = ra.norm_rotary_bwd(x, None, dy, None, w, None, freq, eps=1e-2, interleaved=interleaved, pos_off=1000)
    h = 2.0 ** -7
    for at in ((0, 0, 0, 0), (0, 1, 0, 13), (0, 1, 0, 63), (0, 0, 0, 33)):
        e = torch.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[at])) < 2e-3
    for c in (0, 10, 63):
        e = torch.zeros_like(w)
        e[c] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[c])) < 2e-3


def test_long_rows_and_far_offsets(ra):
    """Rows past 2^31 elements, and angles of positions past 2^40."""
    H, d = 4, 256
    rows = 2 ** 31 // (H * d) + 3
    q = torch.empty(1, rows, H, d, dtype=torch.bfloat16, device="cuda")
    q[:, :2], q[:, -2:] = rand((1, 2, H, d), torch.bfloat16, 21), rand((1, 2, H, d), torch.bfloat16, 22)
    freq = frequencies(d)
    ends = torch.cat((q[:, :2], q[:, -2:]), dim=1)
    want = oracle.rotary(f64(ends), np.array([0, 1, rows - 2, rows - 1]), freq.cpu().numpy())
    ra.ra_rotary_fwd(q, None, freq, q, None)
    got = torch.cat((q[:, :2], q[:, -2:]), dim=1)
    near("ends", got, want, turned_size(f64(ends), freq, False, 1.0), U[torch.bfloat16], 1e-6)
    del q
    # frequencies that are whole fractions of a turn: the angles of far positions are known exactly
    quarter = torch.full((2,), np.pi / 2, dtype=torch.float64, device="cuda")
    x = rand((1, 4, 1, 8), torch.float32, 23)
    y, _ = ra.rotary_fwd(x, None, quarter, pos_off=2 ** 40)
    z, _ = ra.rotary_fwd(x, None, quarter, pos_off=0)
    assert (y - z).abs().max() < 4e-6 * x.abs().max() * 2 ** 40 * 2.0 ** -52 + 1e-3 and torch.isfinite(y).all()


def test_streams_graph_and_other_device(ra):
    B, N, H, d = 2, 300, 4, 64
    q, k = rand((B, N, H, d), torch.bfloat16, 24), rand((B, N, H, d), torch.bfloat16, 25)
    w = rand((d,), torch.bfloat16, 26)
    freq = frequencies(d)
    want = ra.norm_rotary_fwd(q, k, w, w, freq)
    back = ra.norm_rotary_bwd(q, k, q, k, w, w, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ra.norm_rotary_fwd(q, k, w, w, freq, stream=side)
    grads = ra.norm_rotary_bwd(q, k, q, k, w, w, freq, stream=side)
    turned = ra.rotary_fwd(q, k, freq, stream=side)
    side.synchronize()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"] if "address" in b}
    for t in (*got, *grads, *turned):
        assert owner[t.data_ptr()] == side.cuda_stream
    assert all(torch.equal(a, b) for a, b in zip((*got, *grads), (*want, *back)))
    # two captured graphs, each with the workspace it was captured with, replayed in turn on new rows
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = ra.norm_rotary_fwd(q, k, w, w, freq)
            out = ra.norm_rotary_bwd(q, k, y[0], y[1], w, w, freq)
        graphs.append((g, y, out))
    q.copy_(rand((B, N, H, d), torch.bfloat16, 27))
    k.copy_(rand((B, N, H, d), torch.bfloat16, 28))
    y = ra.norm_rotary_fwd(q, k, w, w, freq)
    out = ra.norm_rotary_bwd(q, k, y[0], y[1], w, w, freq)
    for g, *_ in graphs * 2:
        g.replay()
    for _, gy, gout in graphs:
        assert all(torch.equal(a, b) for a, b in zip((*gy, *gout), (*y, *out)))
    with pytest.raises(ra.RAError):
        ra.rotary_fwd(q.cpu(), k.cpu(), freq.cpu())
    with pytest.raises(ra.RAError):
        ra.rotary_fwd(q, k, freq.cpu())
    ra.ra_sync_status()
