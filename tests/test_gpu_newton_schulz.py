"""GPU parity of the Newton-Schulz orthogonalisation against the fp64 oracle.

The operands of the products are fp16, so the distance from the definition is a
few units of 2^-11, amplified or damped by the polynomial's slope at each step.
It is not estimated but computed: `emulate` runs the same formulas in fp64 with
the operands rounded to fp16 where the kernels round them.

One step: what differs between the kernel and `emulate` is fp32 accumulation, at
most K 2^-23 relative per product and near sqrt(K) 2^-24 in the 2-norm (about
3e-6 for K = 2000), and operands that round the other way because of it: a share
of about 2^-11 of them (fp32 noise against fp16 steps) moves by a step of 2^-10,
which adds sqrt(2^-11) 2^-10 < 3e-5 for each of the two products that read such
an operand: 1e-4 covers both.

More steps: the roundings part ways.  A relative difference e between the two
X flips a share e / 2^-10 of the next step's roundings, each by 2^-10, so e
becomes about 2^-10 sqrt(e / 2^-10) = sqrt(2^-10 e), whose fixed point is 2^-10:
from 3e-6 over 5e-5 and 2e-4 to 5e-4 within three steps.  From then on the kernel
and `emulate` are two samples of the same rounding errors, equal in size but not
in sign, so it is their distances from the definition that are compared; a factor
of two leaves room for the few amplified directions that make up most of it.

Both are 2-norms over the matrix, and the output adds half a step of its type.
Sides below 32 average nothing: there single roundings decide, and the bound is
four units of 2^-11 per step, damped by nothing: 20 units, 1e-2."""
import os

import numpy as np
import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

import oracle  # noqa: E402
from tests._parity import f64  # noqa: E402

pytestmark = pytest.mark.gpu

COEFFS = (3.4445, -4.7750, 2.0315)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


def r16(x, scale):
    return (x * scale).astype(np.float16).astype(np.float64) / scale


def emulate(g, steps=5, eps=1e-7, coeffs=COEFFS):
    """The formulas in fp64 with fp16 operands: X as two terms, the Gram matrix
    without the mean of its diagonal."""
    g = np.asarray(g, dtype=np.float64)
    if g.ndim == 3:
        return np.stack([emulate(m, steps, eps, coeffs) for m in g])
    a, b, c = (float(np.float32(v)) for v in coeffs)
    n = np.sqrt(np.square(g).sum()) + eps
    x = g / n if n > 0 else np.zeros_like(g)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    m = x.shape[0]
    sx = 2.0 ** min(14, np.floor(np.log2(np.sqrt(x.size))))
    alpha = 1.0 / m
    for _ in range(steps):
        hi = r16(x, sx)
        x = hi + r16(x - hi, sx)
        a1 = r16(hi @ hi.T - alpha * np.eye(m), 2.0 ** 14)
        b1 = r16((b + 2 * c * alpha) * a1 + c * (a1 @ a1), 2.0 ** 10)
        x = (a + b * alpha + c * alpha * alpha) * x + b1 @ hi
        alpha = np.square(x).sum() / m
    return x.T if tall else x


def rel(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


def gradient(rows, cols, seed, kind="tokens", batch=None):
    """A weight's gradient: a sum over tokens of unequal weight ("tokens"), a plain
    Gaussian, one of low rank under noise, one with decaying singular values."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")

    if batch:
        return torch.stack([gradient(rows, cols, seed * 100 + i, kind) for i in range(batch)])
    if kind == "gauss":
        return randn(rows, cols)
    if kind == "tokens":
        t = 2 * min(rows, cols) + 64
        return (randn(t, rows) * randn(t, 1).exp()).T @ (randn(t, cols) + 0.5 * randn(1, cols)) / t
    k = min(rows, cols)
    if kind == "lowrank":
        r = k // 8 + 1
        return randn(rows, r) @ randn(r, cols) + 0.1 * randn(rows, cols)
    u, _, v = torch.linalg.svd(randn(rows, cols), full_matrices=False)
    return (u * torch.logspace(0, -3, k, device="cuda")) @ v


def check(ra, g, out, steps=5, eps=1e-7, coeffs=COEFFS):
    G, got = f64(g), f64(out)
    assert got.shape == G.shape and np.isfinite(got).all()
    half = HALF[out.dtype]
    for i in range(G.shape[0] if G.ndim == 3 else 1):
        gi, oi = (G[i], got[i]) if G.ndim == 3 else (G, got)
        want, emu = oracle.newton_schulz(gi, coeffs, steps, eps), emulate(gi, steps, eps, coeffs)
        if min(gi.shape) < 32:
            assert rel(oi, want) <= 1e-2 + half, (gi.shape, rel(oi, want))
            continue
        if steps == 1:
            assert rel(oi, emu) <= 1e-4 + half, (gi.shape, rel(oi, emu))
        assert rel(oi, want) <= 2 * rel(emu, want) + 1e-4 + half, (gi.shape, rel(oi, want), rel(emu, want))


SIZES = [(32, 32), (33, 100), (100, 33), (64, 512), (256, 256), (257, 255), (200, 1000), (1000, 333), (130, 3001),
         (768, 520), (1030, 1030),
         # at and around the sizes where the path changes: a side of 128, the other of 64 ... 4096
         (128, 128), (128, 129), (129, 128), (129, 129), (64, 65), (512, 127), (40, 513), (100, 1025), (2049, 128),
         (128, 4096), (128, 4097), (4096, 33), (129, 4096)]


@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(ra, rows, cols):
    for dtype, out in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)):
        g = gradient(rows, cols, rows + cols).to(dtype)
        o = ra.newton_schulz(g, out_dtype=out)
        ra.ra_sync_status()
        check(ra, g, o)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (8, 1), (1, 1000), (2, 3), (5, 40), (17, 300), (31, 31)])
def test_small_sides(ra, rows, cols):
    g = gradient(rows, cols, 3, "gauss")
    o = ra.newton_schulz(g)
    ra.ra_sync_status()
    check(ra, g, o)


@pytest.mark.parametrize("kind", ["gauss", "lowrank", "decay"])
@pytest.mark.parametrize("rows,cols", [(96, 640), (640, 320)])
def test_spectra(ra, kind, rows, cols):
    g = gradient(rows, cols, 21, kind)
    o = ra.newton_schulz(g)
    ra.ra_sync_status()
    check(ra, g, o)


def test_more_tiles_than_pairs(ra):
    g = gradient(2304, 4200, 22, "gauss").bfloat16()
    o = ra.newton_schulz(g, steps=2, out_dtype=torch.float32)
    ra.ra_sync_status()
    check(ra, g, o, steps=2)


@pytest.mark.parametrize("rows,cols", [(128, 300), (300, 128), (513, 770), (1100, 290)])
@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_steps(ra, steps, rows, cols):
    g = gradient(rows, cols, 23)
    o = ra.newton_schulz(g, steps=steps)
    ra.ra_sync_status()
    check(ra, g, o, steps=steps)


def test_other_coefficients(ra):
    # the cubic (3/2, -1/2, 0) and a quintic that ends at one
    g = gradient(64, 200, 24, "gauss")
    for coeffs, steps in (((1.5, -0.5, 0.0), 4), ((1.875, -1.25, 0.375), 6)):
        o = ra.newton_schulz(g, steps=steps, coeffs=coeffs)
        ra.ra_sync_status()
        want = oracle.newton_schulz(f64(g), coeffs, steps)
        assert rel(f64(o), want) <= 2e-3


@pytest.mark.parametrize("rows,cols", [(40, 96), (300, 130), (96, 1500)])
def test_batch_equals_single_matrices(ra, rows, cols):
    g = gradient(rows, cols, 25, batch=5)
    g[2] *= 1e4
    g[3] *= 1e-4
    o = ra.newton_schulz(g)
    ra.ra_sync_status()
    check(ra, g, o)
    for i in range(5):
        assert torch.equal(o[i], ra.newton_schulz(g[i])), i


@pytest.mark.parametrize("rows,cols", [(100, 77), (150, 177), (77, 300)])
def test_strides_and_in_place(ra, rows, cols):
    g = gradient(rows, cols, 26, batch=3)
    want = ra.newton_schulz(g)
    wide = torch.full((3, rows + 10, cols + 13), float("nan"), device="cuda")
    wide[:, 5:5 + rows, 3:3 + cols] = g
    view = wide[:, 5:5 + rows, 3:3 + cols]
    assert torch.equal(ra.newton_schulz(view), want)
    ws = torch.empty(ra.ra_newton_schulz_workspace_bytes(3, rows, cols), dtype=torch.uint8, device="cuda")
    ra.ra_newton_schulz(view, view, ws)        # in place, in a larger tensor
    ra.ra_sync_status()
    assert torch.equal(view, want)
    wide[:, 5:5 + rows, 3:3 + cols] = float("nan")
    assert torch.isnan(wide).all()             # nothing written beside it


@pytest.mark.parametrize("rows,cols", [(64, 96), (140, 200)])
def test_scale_of_the_gradient(ra, rows, cols):
    # powers of two change nothing but the norm's last bit (its squares are summed by
    # magnitude), from norms whose squares overflow or vanish in fp32 to ordinary ones
    g = gradient(rows, cols, 27)
    want = f64(ra.newton_schulz(g, steps=1, eps=0.0))
    for k in (-100, -70, -30, 30, 62, 100):
        o = ra.newton_schulz(g * 2.0 ** k, steps=1, eps=0.0)
        assert rel(f64(o), want) <= 1e-4, k
        check(ra, g * 2.0 ** k, ra.newton_schulz(g * 2.0 ** k, eps=0.0), eps=0.0)
    ra.ra_sync_status()


@pytest.mark.parametrize("rows,cols", [(40, 50), (150, 140)])
def test_zero_and_unusable_gradients(ra, rows, cols):
    z = torch.zeros(2, rows, cols, device="cuda")
    for eps in (1e-7, 0.0):
        assert not ra.newton_schulz(z, eps=eps).any()
    g = gradient(rows, cols, 28, batch=3)
    good = ra.newton_schulz(g)
    g[1, 3, 4] = float("nan")
    o = ra.newton_schulz(g)
    assert torch.isnan(o[1]).all() and torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    g[1, 3, 4] = float("inf")
    o = ra.newton_schulz(g)
    ra.ra_sync_status()
    assert torch.isnan(o[1]).any() and torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])


@pytest.mark.parametrize("rows,cols", [(300, 700), (100, 2000)])
def test_repeats_and_other_streams(ra, rows, cols):
    g = gradient(rows, cols, 29, batch=2)
    want = ra.newton_schulz(g)
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            outs.append(ra.newton_schulz(g, stream=s))
    torch.cuda.synchronize()
    ra.ra_sync_status()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("rows,cols", [(200, 520), (120, 520)])
def test_replays_from_a_cuda_graph(ra, rows, cols):
    g = gradient(rows, cols, 30)
    out = torch.empty_like(g)
    ws = torch.empty(ra.ra_newton_schulz_workspace_bytes(1, rows, cols), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    ra.ra_newton_schulz(g, out, ws, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ra.ra_newton_schulz(g, out, ws, stream=stream)
    g.copy_(gradient(rows, cols, 31))
    out.fill_(float("nan"))
    ws.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    ra.ra_sync_status()
    assert torch.equal(out, ra.newton_schulz(g))


@pytest.mark.parametrize("rows,cols", [(131, 77), (131, 177), (77, 131)])
def test_nothing_is_written_past_the_buffers(ra, rows, cols):
    guard = 4096
    g = gradient(rows, cols, 32)
    buf = torch.full((rows * cols + 2 * guard,), 7.0, device="cuda")
    n = ra.ra_newton_schulz_workspace_bytes(1, rows, cols)
    ws = torch.full((n + guard,), 9, dtype=torch.uint8, device="cuda")
    ra.ra_newton_schulz(g, buf[guard:guard + rows * cols].view(rows, cols), ws[:n])
    ra.ra_sync_status()
    assert (buf[:guard] == 7).all() and (buf[guard + rows * cols:] == 7).all() and (ws[n:] == 9).all()


@pytest.mark.parametrize("batch,rows,cols", [(1, 100, 1757), (2, 2048, 128), (12, 128, 2000), (40, 65, 513), (3, 1, 2049)])
def test_slices_of_small_matrices(ra, batch, rows, cols):
    # slices of 64, 128 and 256 columns, as size and batch ask for
    g = torch.stack([gradient(rows, cols, 50 + i, "gauss") for i in range(batch)])
    o = ra.newton_schulz(g)
    ra.ra_sync_status()
    check(ra, g, o)
