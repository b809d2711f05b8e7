"""The operators of a training step run together, as a trainer calls them: the
feed-forward layer, the vocabulary cross entropy of its output, the gradients
back through both, and the orthogonalised updates of the layer's two matrices;
eager and captured into a CUDA graph.

Every stage is checked against the fp64 oracle on the values that stage was
given, within the bounds of its own tests; that the stages' oracles compose to
the gradient of the whole is checked on the CPU by finite differences."""
import os

import numpy as np
import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

import oracle  # noqa: E402
from tests import test_gpu_newton_schulz as ns  # noqa: E402
from tests import test_gpu_xent as xe  # noqa: E402
from tests._parity import f64  # noqa: E402

T, DM, DH, V = 384, 256, 768, 2000


def test_oracles_compose_to_the_gradient_of_the_whole():
    rng = np.random.default_rng(5)
    t, dm, dh, v = 5, 4, 8, 11
    x, w1, w2, wv = (rng.standard_normal(s) for s in ((t, dm), (dh, dm), (dm, dh), (v, dm)))
    y, g = rng.integers(0, v, t), rng.random(t)
    y[1] = -100

    def total(w1_, w2_, wv_):
        return float(oracle.xent_fwd(oracle.ffn_fwd(x, w1_, w2_)[0], wv_, y)[0] @ g)

    out = oracle.ffn_fwd(x, w1, w2)[0]
    dout, dwv, _ = oracle.xent_bwd(out, wv, y, g)
    _, dw1, dw2, _ = oracle.ffn_bwd(x, w1, w2, dout)
    eps = 1e-6
    for i, (m, grad) in enumerate(((w1, dw1), (w2, dw2), (wv, dwv))):
        fd = np.zeros_like(m)
        for j in np.ndindex(m.shape):
            hi, lo = [w1, w2, wv], [w1, w2, wv]
            hi[i], lo[i] = m.copy(), m.copy()
            hi[i][j] += eps
            lo[i][j] -= eps
            fd[j] = (total(*hi) - total(*lo)) / (2 * eps)
        np.testing.assert_allclose(grad, fd, rtol=1e-5, atol=1e-8)


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


def inputs(dtype, seed):
    from blockwise_exact_attention_ra_gb300.inputs import make_ffn
    x, w1, w2, _ = make_ffn(T, DM, DH, dtype, "cuda", seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    wv = (torch.randn(V, DM, generator=gen, device="cuda") * DM ** -0.5).to(dtype)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    y[::7] = -100
    g = torch.full((T,), (256.0 if dtype == torch.float16 else 1.0) / T, device="cuda")
    return x, w1, w2, wv, y, g


def step(ra, x, w1, w2, wv, y, g, stream=None):
    out = ra.ffn_fwd(x, w1, w2, 128, stream=stream)
    loss, lse = ra.xent_fwd(out, wv, y, stream=stream)
    dout, dwv = ra.xent_bwd(out, wv, y, lse, g, dx_dtype=x.dtype, dw_dtype=x.dtype, stream=stream)
    _, dw1, dw2 = ra.ffn_bwd(x, w1, w2, dout, 128, stream=stream)
    return out, loss, lse, dout, dwv, dw1, dw2, ra.newton_schulz(dw1, out_dtype=x.dtype, stream=stream), \
        ra.newton_schulz(dw2, out_dtype=x.dtype, stream=stream)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step(ra, dtype):
    x, w1, w2, wv, y, g = inputs(dtype, 41)
    out, loss, lse, dout, dwv, dw1, dw2, u1, u2 = step(ra, x, w1, w2, wv, y, g)
    ra.ra_sync_status()
    xe.check(ra, out, wv, y, g, loss, lse, dout, dwv)
    X, W1, W2, D = f64(x), f64(w1), f64(w2), f64(dout)
    _, r1, r2, _ = oracle.ffn_bwd(X, W1, W2, D)
    h = X @ W1.T
    a, dh = oracle.gelu(h), (D @ W2) * oracle.gelu_grad(h)
    u = xe.U[dtype]
    # GELU(h) carries one rounding; dH those of GELU'(h) and its own; fp32 sums of T products
    for name, got, want, bound in (("dw2", dw2, r2, (u + T * 2.0 ** -24) * (np.abs(D).T @ np.abs(a))),
                                   ("dw1", dw1, r1, (2.1 * u + T * 2.0 ** -24) * (np.abs(dh).T @ np.abs(X)))):
        assert float((np.abs(f64(got) - want) - bound).max()) <= 1e-6 * np.abs(want).max(), name
    ns.check(ra, dw1, u1)
    ns.check(ra, dw2, u2)


@pytest.mark.gpu
def test_step_replays_from_a_cuda_graph_beside_an_eager_one(ra):
    first, second = inputs(torch.bfloat16, 42), inputs(torch.bfloat16, 43)
    want = [step(ra, *first), step(ra, *second)]
    held = [t.clone() for t in first]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step(ra, *held, stream=stream)
    for i, src in enumerate((first, second, first)):
        for h, s in zip(held, src):
            h.copy_(s)
        graph.replay()
        eager = step(ra, *second)            # with workspaces of its own, on another stream
        torch.cuda.synchronize()
        ra.ra_sync_status()
        for a, b in zip(got, want[i % 2]):
            assert torch.equal(a, b)
        for a, b in zip(eager, want[1]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_what_a_call_on_another_stream_allocates_belongs_to_that_stream(ra):
    """Or the allocator could hand a workspace, freed when the call returns, to work of the
    current stream while the kernels still use it."""
    x, w1, w2, wv, y, g = inputs(torch.bfloat16, 44)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    loss, lse = ra.xent_fwd(x, wv, y, stream=stream)
    dx, dw = ra.xent_bwd(x, wv, y, lse, g, stream=stream)
    u = ra.newton_schulz(w1, stream=stream)
    stream.synchronize()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"] if "address" in b}
    for t in (loss, lse, dx, dw, u):
        assert owner[t.data_ptr()] == stream.cuda_stream
