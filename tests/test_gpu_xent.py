"""GPU parity of the vocabulary cross entropy (loss, lse, dx, dw) against the
fp64 oracle.

Tolerances follow from the arithmetic.  With s_t = max_v sum_k |x_tk w_vk|:
  logits: fp32 accumulation of D exact products, at most D 2^-23 s_t (the tensor
    core may truncate);
  lse: that, the rounding of the exponent's argument (|z| log2(e) 2^-24, twice),
    the exponential's and the sums' relative errors (2^-22 + 2^-19 for sums of up
    to a few hundred parts of up to 128 terms in four chains), and lse's own
    rounding: e_lse = D 2^-23 s + 2^-21 max|z| + 2^-18 + 2^-23 |lse|;
  loss: e_lse + D 2^-23 s;
  d = g (p - [v = y]): |dloss| p (e_z + e_lse) and half a unit of the operand
    type, u = 2^-8 (bf16) or 2^-11 (fp16; its subnormals add g_max 2^-38);
    probabilities below 2^-126, fp32's smallest normal number, may become zero, and
    so may gradients below it: (1 + |dloss|) 2^-126;
  dx, dw: the sum of |error of d| times the other factor, K 2^-23 of the absolute
    products, and half a unit of the output type."""
import os

import numpy as np
import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

import oracle  # noqa: E402
from tests._parity import f64  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


def make(T, D, V, dtype, seed, ignored=0.25, scale=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    w = torch.randn(V, D, generator=gen, device="cuda") * (1.5 * scale / D ** 0.5)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    x = torch.randn(T, D, generator=gen, device="cuda")
    x += 8 * torch.rand(T, 1, generator=gen, device="cuda") * w[y] / w[y].norm(dim=1, keepdim=True)
    drop = torch.rand(T, generator=gen, device="cuda") < ignored
    y = torch.where(drop, torch.full_like(y, -100), y)
    g = (0.5 + torch.rand(T, generator=gen, device="cuda")) * (16.0 if dtype == torch.float16 else 1.0 / T)
    return x.to(dtype), w.to(dtype), y, g


def within(name, got, want, bound):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    worst = float((np.abs(got - want) - bound).max())
    assert worst <= 0.0, f"{name}: past its bound by {worst:.3e} (max err {np.abs(got - want).max():.3e})"


def check(ra, x, w, y, g, loss, lse, dx=None, dw=None):
    X, W, Y, G = f64(x), f64(w), y.cpu().numpy(), f64(g)
    T, D = X.shape
    r_loss, r_lse, z = oracle.xent_fwd(X, W, Y)
    s = (np.abs(X) @ np.abs(W).T).max(axis=1)
    e_z = D * 2.0 ** -23 * s
    e_lse = e_z + 2.0 ** -21 * np.abs(z).max(axis=1) + 2.0 ** -18 + 2.0 ** -23 * np.abs(r_lse)
    within("lse", f64(lse), r_lse, e_lse)
    kept = Y != -100
    within("loss", f64(loss), r_loss, np.where(kept, e_lse + e_z, 0.0))
    if dx is None:
        return
    r_dx, r_dw, d = oracle.xent_bwd(X, W, Y, G)
    p = np.exp(z - r_lse[:, None])
    u = U[x.dtype]
    live = np.where(kept, np.abs(G), 0.0)
    e_d = live[:, None] * p * (e_z + e_lse)[:, None] * 1.01 + 1.01 * u * np.abs(d)
    e_d = e_d + (1.0 + live[:, None]) * 2.0 ** -126
    if x.dtype == torch.float16:
        e_d = e_d + live.max() * 2.0 ** -38
    e_d[~kept] = 0.0
    V = W.shape[0]
    for name, got, want, bound in (
            ("dx", dx, r_dx, e_d @ np.abs(W) + V * 2.0 ** -23 * (np.abs(d) @ np.abs(W))),
            ("dw", dw, r_dw, e_d.T @ np.abs(X) + T * 2.0 ** -23 * (np.abs(d).T @ np.abs(X)))):
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0   # half a subnormal step of the output
        within(name, f64(got), want, bound + U[got.dtype] * (np.abs(want) + bound) + tiny)


SIZES = [
    # T, D, V, block
    (1, 8, 1, 1), (1, 64, 1000, 256), (2, 2048, 3000, 1024), (3, 72, 5, 2), (4, 264, 20011, 8192), (7, 2048, 333, 333),
    (8, 2040, 700, 256), (8, 2056, 700, 256), (9, 64, 2001, 500), (127, 64, 255, 255), (128, 128, 256, 128), (129, 136, 257, 100),
    (256, 200, 1025, 512), (333, 256, 2000, 768), (600, 520, 1111, 1111), (1025, 64, 3001, 1024), (40, 1048, 777, 256),
]


@pytest.mark.parametrize("T,D,V,block", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_sizes(ra, T, D, V, block, dtype):
    x, w, y, g = make(T, D, V, dtype, 7 * T + V)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=block)
    dx16, dw16 = ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=dtype, dw_dtype=dtype)
    ra.ra_sync_status()
    check(ra, x, w, y, g, loss, lse, dx, dw)
    check(ra, x, w, y, g, loss, lse, dx16, dw16)


def test_many_tiles(ra):
    # more tiles than CTA pairs in every product, several blocks, mixed output types
    x, w, y, g = make(2304, 320, 9000, torch.bfloat16, 5)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=4096, dx_dtype=torch.bfloat16, dw_dtype=torch.float16)
    ra.ra_sync_status()
    check(ra, x, w, y, g, loss, lse, dx, dw)


def check_on_gpu(x, w, y, g, loss, lse, dx, dw):
    """`check` for sizes at which the CPU's fp64 takes too long: the same formulas and
    bounds in fp64 torch operations on the GPU."""
    X, W, G = x.double(), w.double(), g.double()
    (T, D), V = X.shape, W.shape[0]
    z = X @ W.T
    r_lse = torch.logsumexp(z, dim=1)
    kept = y != -100
    at = torch.where(kept, y, torch.zeros_like(y))[:, None]
    s = (X.abs() @ W.abs().T).amax(dim=1)
    e_z = D * 2.0 ** -23 * s
    e_lse = e_z + 2.0 ** -21 * z.abs().amax(dim=1) + 2.0 ** -18 + 2.0 ** -23 * r_lse.abs()
    zero = torch.zeros_like(r_lse)

    def inside(name, got, want, bound):
        worst = float(((got.double() - want).abs() - bound).max())
        assert worst <= 0.0, f"{name}: past its bound by {worst:.3e}"
    inside("lse", lse, r_lse, e_lse)
    inside("loss", loss, torch.where(kept, r_lse - z.gather(1, at)[:, 0], zero), torch.where(kept, e_lse + e_z, zero))
    live = torch.where(kept, G, zero)
    p = torch.exp(z - r_lse[:, None])
    d = p.clone()
    d.scatter_add_(1, at, torch.full_like(r_lse, -1.0)[:, None])
    d *= live[:, None]
    e_d = live.abs()[:, None] * p * (e_z + e_lse)[:, None] * 1.01 + 1.01 * U[x.dtype] * d.abs()
    e_d += (1.0 + live.abs()[:, None]) * 2.0 ** -126
    if x.dtype == torch.float16:
        e_d += live.abs().max() * 2.0 ** -38
    e_d *= kept[:, None]
    for name, got, want, bound in (
            ("dx", dx, d @ W, e_d @ W.abs() + V * 2.0 ** -23 * (d.abs() @ W.abs())),
            ("dw", dw, d.T @ X, e_d.T @ X.abs() + T * 2.0 ** -23 * (d.abs().T @ X.abs()))):
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
        inside(name, got, want, bound + U[got.dtype] * (want.abs() + bound) + tiny)


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
def test_several_blocks(ra, dtype, out):
    # blocks of more than 256 MB of gradient (2 x 4100 entries, the last of 200): dx summed
    # over them in fp32, in the workspace or in dx itself
    T, D, V, block = 33000, 72, 8400, 4100
    assert 2 * T * block > 256 << 20
    x, w, y, g = make(T, D, V, dtype, 6)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=out, dw_dtype=out)
    ra.ra_sync_status()
    check_on_gpu(x, w, y, g, loss, lse, dx, dw)


def test_several_blocks_with_split_products(ra):
    # few tiles of dx and long blocks: K of dx = d W is split, its planes summed over blocks;
    # the last block (100) is too short for as many splits
    T, D, V, block = 4200, 8, 64300, 32100
    assert 2 * T * block > 256 << 20
    x, w, y, g = make(T, D, V, torch.bfloat16, 17)
    loss, lse = ra.xent_fwd(x, w, y)
    for out in (torch.bfloat16, torch.float32):
        dx, dw = ra.xent_bwd(x, w, y, lse, g, block=block, dx_dtype=out, dw_dtype=out)
        ra.ra_sync_status()
        check_on_gpu(x, w, y, g, loss, lse, dx, dw)


def test_checks_on_cpu_and_gpu_agree(ra):
    x, w, y, g = make(90, 64, 300, torch.float16, 18)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g)
    check(ra, x, w, y, g, loss, lse, dx, dw)
    check_on_gpu(x, w, y, g, loss, lse, dx, dw)
    # a mistake planted in what the oracle is told is past the bounds of both
    g2 = g.clone()
    g2[int(torch.nonzero(y != -100)[0])] *= 1.1
    for f in (lambda: check(ra, x, w, y, g2, loss, lse, dx, dw), lambda: check_on_gpu(x, w, y, g2, loss, lse, dx, dw)):
        with pytest.raises(AssertionError):
            f()


def test_row_strides(ra):
    x, w, y, g = make(200, 128, 700, torch.bfloat16, 11)
    wide_x = torch.full((200, 3, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_w = torch.full((700, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[:, 1], wide_w[:, :128] = x, w
    xs, ws = wide_x[:, 1], wide_w[:, :128]
    a, b = ra.xent_fwd(x, w, y), ra.xent_fwd(xs, ws, y)
    ga, gb = ra.xent_bwd(x, w, y, a[1], g, block=256), ra.xent_bwd(xs, ws, y, b[1], g, block=256)
    ra.ra_sync_status()
    for p, q in zip(a + ga, b + gb):
        assert torch.equal(p, q)


def test_all_tokens_ignored(ra):
    x, w, y, g = make(70, 64, 300, torch.bfloat16, 3)
    y = torch.full_like(y, -100)
    g = torch.full_like(g, float("nan"))      # not used at ignored tokens
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=128)
    ra.ra_sync_status()
    assert not loss.any() and torch.isfinite(lse).all() and not dx.any() and not dw.any()


def test_ignored_token_with_unusable_values(ra):
    # NaN and infinities in a token without loss reach neither dx nor its own row's
    # gradient; dw multiplies them by an exact zero, as the formula does
    x, w, y, g = make(130, 64, 300, torch.bfloat16, 4, ignored=0.0)
    y[5] = -100
    ref = ra.xent_fwd(x, w, y)
    rdx, _ = ra.xent_bwd(x, w, y, ref[1], g, block=128)
    x2 = x.clone()
    x2[5] = float("inf")
    loss, lse = ra.xent_fwd(x2, w, y)
    dx, _ = ra.xent_bwd(x2, w, y, lse, g, block=128)
    ra.ra_sync_status()
    assert torch.equal(loss, ref[0]) and torch.equal(dx, rdx)


def test_other_ignore_index(ra):
    x, w, y, g = make(90, 64, 300, torch.float16, 6)
    y7 = torch.where(y == -100, torch.full_like(y, 7), torch.where(y == 7, torch.full_like(y, 8), y))
    y100 = torch.where(y == 7, torch.full_like(y, 8), y)
    a, b = ra.xent_fwd(x, w, y7, ignore_index=7), ra.xent_fwd(x, w, y100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for p, q in zip(ra.xent_bwd(x, w, y7, a[1], g, ignore_index=7), ra.xent_bwd(x, w, y100, b[1], g)):
        assert torch.equal(p, q)
    ra.ra_sync_status()


def test_target_outside_the_vocabulary(ra):
    x, w, y, g = make(64, 64, 300, torch.bfloat16, 8, ignored=0.0)
    good = ra.xent_fwd(x, w, y)
    for bad in (300, -1, 2 ** 40, -2 ** 62):
        y2 = y.clone()
        y2[9] = bad
        loss, lse = ra.xent_fwd(x, w, y2)
        with pytest.raises(ra.RAError) as e:
            ra.ra_sync_status()
        assert e.value.code == 1 and "vocabulary" in str(e.value)
        assert torch.isnan(loss[9]) and torch.equal(lse, good[1])
        keep = torch.arange(64, device="cuda") != 9
        assert torch.equal(loss[keep], good[0][keep])
        dx, dw = ra.xent_bwd(x, w, y2, lse, g)
        ra.ra_sync_status()
        assert not dx[9].any() and torch.isfinite(dw).all()


def test_large_logits(ra):
    # logits of several hundred: the maximum is taken out before the exponentials
    x, w, y, g = make(150, 64, 500, torch.bfloat16, 9, scale=60.0)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=256)
    ra.ra_sync_status()
    check(ra, x, w, y, g, loss, lse, dx, dw)


def test_infinite_logits(ra):
    x, w, y, _ = make(40, 64, 300, torch.bfloat16, 10, ignored=0.0)
    x[:, 0], w[:, 0] = 1.0, 0.0
    ref, rl = ra.xent_fwd(x, w, y)
    w2 = w.clone()
    dead = (int(y[3]) + 1) % 300
    w2[dead, 0] = float("-inf")               # one entry that no token can take
    loss, lse = ra.xent_fwd(x, w2, y)
    W = f64(w2)
    W[dead, 0] = -1e4
    want, wl, _ = oracle.xent_fwd(f64(x), W, y.cpu().numpy())
    other = y.cpu().numpy() != dead
    np.testing.assert_allclose(f64(loss)[other], want[other], atol=1e-4)
    assert torch.isinf(loss[torch.from_numpy(~other).cuda()]).all()
    w2[:, 0] = float("-inf")                  # no entry left
    loss, lse = ra.xent_fwd(x, w2, y)
    assert torch.isinf(lse).all() and (lse < 0).all() and torch.isnan(loss).all()
    w2[:, 0] = float("nan")
    loss, lse = ra.xent_fwd(x, w2, y)
    ra.ra_sync_status()
    assert torch.isnan(lse).all() and torch.isnan(loss).all()


def test_small_and_large_gradients_of_the_loss_in_fp16(ra):
    # the operand's power of two follows max |dloss|: 2^-30 and 2^30 give the same bits
    x, w, y, g = make(100, 64, 400, torch.float16, 12)
    _, lse = ra.xent_fwd(x, w, y)
    a = ra.xent_bwd(x, w, y, lse, g)
    for k in (-30, 30):
        b = ra.xent_bwd(x, w, y, lse, g * 2.0 ** k)
        for p, q in zip(a, b):
            assert torch.equal(p, q * 2.0 ** -k)
    ra.ra_sync_status()


def test_repeats_and_other_streams(ra):
    x, w, y, g = make(700, 256, 5000, torch.bfloat16, 13)
    a = ra.xent_fwd(x, w, y)
    ga = ra.xent_bwd(x, w, y, a[1], g, block=2048, dx_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:                          # two calls at once, each with its own workspace
        with torch.cuda.stream(s):
            b = ra.xent_fwd(x, w, y, stream=s)
            outs.append(b + ra.xent_bwd(x, w, y, b[1], g, block=2048, dx_dtype=torch.bfloat16, stream=s))
    torch.cuda.synchronize()
    ra.ra_sync_status()
    for b in outs:
        for p, q in zip(a + ga, b):
            assert torch.equal(p, q)


def test_replays_from_a_cuda_graph(ra):
    x, w, y, g = make(300, 128, 3000, torch.float16, 14)
    T, D, V = 300, 128, 3000
    loss, lse = (torch.empty(T, device="cuda") for _ in range(2))
    dx, dw = torch.empty(T, D, dtype=torch.float16, device="cuda"), torch.empty(V, D, device="cuda")
    wf = torch.empty(ra.ra_xent_fwd_workspace_bytes(ra.RA_F16, T, D, V), dtype=torch.uint8, device="cuda")
    wb = torch.empty(ra.ra_xent_bwd_workspace_bytes(ra.RA_F16, ra.RA_F16, T, D, V, 1024), dtype=torch.uint8,
                     device="cuda")
    stream = torch.cuda.Stream()

    def step():
        ra.ra_xent_fwd(x, w, y, loss, lse, wf, stream=stream)
        ra.ra_xent_bwd(x, w, y, lse, g, 1024, dx, dw, wb, stream=stream)

    stream.wait_stream(torch.cuda.current_stream())
    step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    x2, _, y2, g2 = make(T, D, V, torch.float16, 15)
    for t, s in ((x, x2), (y, y2), (g, g2)):
        t.copy_(s)
    for t in (loss, lse, dx, dw):
        t.fill_(float("nan"))
    wf.fill_(255)
    wb.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    ra.ra_sync_status()
    a = ra.xent_fwd(x, w, y)
    ga = ra.xent_bwd(x, w, y, a[1], g, block=1024, dx_dtype=torch.float16)
    for p, q in zip(a + ga, (loss, lse, dx, dw)):
        assert torch.equal(p, q)


def test_nothing_is_written_past_the_outputs(ra):
    T, D, V = 131, 72, 517
    x, w, y, g = make(T, D, V, torch.bfloat16, 16)
    guard = 4096

    def guarded(n, dtype):
        t = torch.full((n + 2 * guard,), 7.0, dtype=dtype, device="cuda")
        return t, t[guard:guard + n]

    lo, loss = guarded(T, torch.float32)
    le, lse = guarded(T, torch.float32)
    dxb, dx = guarded(T * D, torch.bfloat16)
    dwb, dw = guarded(V * D, torch.bfloat16)
    nf = ra.ra_xent_fwd_workspace_bytes(ra.RA_BF16, T, D, V)
    nb = ra.ra_xent_bwd_workspace_bytes(ra.RA_BF16, ra.RA_BF16, T, D, V, 200)
    wf = torch.full((nf + guard,), 9, dtype=torch.uint8, device="cuda")
    wb = torch.full((nb + guard,), 9, dtype=torch.uint8, device="cuda")
    ra.ra_xent_fwd(x, w, y, loss, lse, wf[:nf])
    ra.ra_xent_bwd(x, w, y, lse, g, 200, dx.view(T, D), dw.view(V, D), wb[:nb])
    ra.ra_sync_status()
    for b, n in ((lo, T), (le, T), (dxb, T * D), (dwb, V * D)):
        assert (b[:guard] == 7).all() and (b[guard + n:] == 7).all()
    assert (wf[nf:] == 9).all() and (wb[nb:] == 9).all()
    check(ra, x, w, y, g, loss, lse, dx.view(T, D), dw.view(V, D))


FEW = [
    # T, D, V: ends of units of 16 entries and of rounds of them (152 blocks, four at a time), sums in
    # several pieces, the longest rows that x's share of shared memory holds and the first past it
    (2, 40, 15), (5, 72, 16), (9, 32, 17), (16, 8, 9729), (10, 264, 64), (3, 4104, 200), (8, 13408, 40), (8, 13448, 40),
    (16, 5664, 65), (16, 5672, 65), (17, 64, 700),
]


@pytest.mark.parametrize("T,D,V", FEW)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_few_tokens(ra, T, D, V, dtype):
    x, w, y, g = make(T, D, V, dtype, T + D + V)
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g)
    ra.ra_sync_status()
    check(ra, x, w, y, g, loss, lse, dx, dw)


def test_few_tokens_with_strides_and_unusable_values(ra):
    x, w, y, g = make(12, 72, 500, torch.bfloat16, 31, ignored=0.0)
    wide_x = torch.full((12, 3, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_w = torch.full((500, 88), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[:, 1], wide_w[:, :72] = x, w
    y[3], y[7] = -100, 500                     # no loss; outside the vocabulary
    g[3] = g[7] = float("nan")
    loss, lse = ra.xent_fwd(wide_x[:, 1], wide_w[:, :72], y)
    with pytest.raises(ra.RAError):
        ra.ra_sync_status()
    dx, dw = ra.xent_bwd(wide_x[:, 1], wide_w[:, :72], y, lse, g)
    ra.ra_sync_status()
    assert torch.isnan(loss[7]) and not dx[3].any() and not dx[7].any()
    y[7], g[3], g[7] = -100, 0.0, 0.0
    loss[7] = 0.0
    check(ra, x, w, y, g, loss, lse, dx, dw)


def test_few_tokens_in_several_blocks(ra):
    T, D, V, block = 16, 8, 9000000, 8500000
    assert 2 * T * block > 256 << 20
    x, w, y, g = make(T, D, V, torch.float16, 32)
    y[0], y[1] = block - 2, block + 1          # targets beside the blocks' edge
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g, block=block)
    ra.ra_sync_status()
    check_on_gpu(x, w, y, g, loss, lse, dx, dw)


@pytest.mark.parametrize("T,D,V", [(1, 64, 700), (2, 2048, 20011), (16, 264, 1000), (17, 72, 300), (40, 1048, 9000),
                                   (64, 136, 5001), (64, 9800, 130)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_few_tokens_lose_nothing_to_the_rounding_of_the_logit_gradients(ra, T, D, V, dtype):
    """Up to 64 tokens d is kept as two terms: its error is u^2 instead of the u that `check`
    allows (dx whole and split, its tiles' rows full and not)."""
    x, w, y, g = make(T, D, V, dtype, 3 * T + V, ignored=0.0)
    _, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g)
    ra.ra_sync_status()
    X, W, G = x.double(), w.double(), g.double()
    z = X @ W.T
    e_z = D * 2.0 ** -23 * (X.abs() @ W.abs().T).amax(dim=1)
    e_lse = e_z + 2.0 ** -21 * z.abs().amax(dim=1) + 2.0 ** -18 + 2.0 ** -23 * torch.logsumexp(z, 1).abs()
    p = torch.softmax(z, dim=1)
    d = p.clone()
    d[torch.arange(T), y] -= 1.0
    d *= G[:, None]
    u = U[dtype]
    # as in `check`; d itself is an fp32 number (2^-22: the difference and the product)
    e_d = G.abs()[:, None] * p * (e_z + e_lse)[:, None] * 1.01 + (1.01 * u * u + 2.0 ** -22) * d.abs()
    e_d += (1.0 + G.abs()[:, None]) * 2.0 ** -126 + (G.abs().max() * 2.0 ** -38 if dtype == torch.float16 else 0.0)
    for name, got, want, bound in (
            ("dx", dx, d @ W, e_d @ W.abs() + 2 * V * 2.0 ** -23 * (d.abs() @ W.abs())),
            ("dw", dw, d.T @ X, e_d.T @ X.abs() + 2 * T * 2.0 ** -23 * (d.abs().T @ X.abs()))):
        worst = float(((got.double() - want).abs() - bound - U[torch.float32] * want.abs()).max())
        assert worst <= 0.0, f"{name}: past its bound by {worst:.3e}"
