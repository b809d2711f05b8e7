"""The global norm of many tensors and clipping by it, on the GPU, against fp64.

Tolerances.  Squares are exact to 2^-24 each and summed over at most 64 elements in fp32 (two
chains of 32 and their sum: 33 x 2^-24 of a sum of positive terms), then in fp64; the root halves
it and its rounding to fp32 adds 2^-24: 1.1e-6 in all.  The factor carries the same, its rounding
and the product's 2^-24 each, and the result half a step u of its type."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests._parity import f64

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu
NORM, MUL = 1.2e-6, 1.4e-6  # (33 / 2 + 1) 2^-24 = 1.05e-6, and two roundings more


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


def tensors(sizes, types, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(t) for n, t in zip(sizes, types)]


def check(ra, grads, max_norm, outs=None, eps=1e-6):
    """One call into new tensors and one in place, against fp64."""
    want = oracle.global_norm([f64(t) for t in grads])
    c = oracle.clip_factor(want, float(np.float32(max_norm)), float(np.float32(eps)))
    kept = [t.clone() for t in grads]
    n0 = ra.grad_norm(grads)
    outs = [torch.full_like(t, 7) for t in grads] if outs is None else outs
    n1 = ra.grad_clip(grads, max_norm, outs=outs, eps=eps)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    n2 = ra.grad_clip(grads, max_norm, eps=eps)
    ra.ra_sync_status()
    assert n0.shape == () and float(n0) == float(n1) == float(n2)
    if want > torch.finfo(torch.float32).max:  # 2e37 x 273: no fp32 number; the factor has to be right all the same
        assert float(n0) == float("inf")
    else:
        assert abs(float(n0) - want) <= NORM * want + 2.0 ** -149
    for t, k, o in zip(grads, kept, outs):
        x = f64(k) * c
        for y in (t, o):
            step = torch.finfo(y.dtype)
            lim = (step.eps / 2 * 1.001 + MUL) * np.abs(x) + step.smallest_normal * step.eps / 2
            assert (np.abs(f64(y) - x) <= lim).all()
        if c == 1.0:
            assert torch.equal(t, k)


F, H, Bf = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
@pytest.mark.parametrize("sizes,types", [
    ([1], [F]), ([7], [Bf]), ([8], [H]), ([2047, 2048, 2049, 4097], [F, Bf, H, Bf]), ([100003], [F]),
    ([0, 5, 0, 3], [F, F, Bf, H]), ([1 << 20, 33, 1, 12345], [Bf, F, H, F]), ([3000001], [Bf]),
])
def test_sizes_and_types(ra, sizes, types, max_norm):
    check(ra, tensors(sizes, types, 1), max_norm)


@pytest.mark.parametrize("count", [47, 48, 49, 1023, 1024, 1025, 2500])
def test_many_tensors(ra, count):
    """Up to a launch's number of tensors and past it."""
    sizes = [(i * 37) % 300 for i in range(count)]
    check(ra, tensors(sizes, [(F, Bf, H)[i % 3] for i in range(count)], 2), 1.0)


@pytest.mark.parametrize("dtype", [F, Bf, H])
def test_views_at_any_offset(ra, dtype):
    """Views of a flat buffer that start between 16-byte boundaries, into outputs that lie as they do
    and otherwise; what lies between the views stays as it was."""
    flat = tensors([60000], [dtype], 3)[0]
    cuts = [(1, 5), (7, 3000), (3001, 9000), (9001, 9001), (9003, 40000), (40003, 59999)]
    for shift, to in ((0, dtype), (1, dtype), (3, F), (1, Bf), (2, H)):
        buf = torch.full((60010,), 3.0, device="cuda", dtype=to)
        outs = [buf[a + shift:b + shift] for a, b in cuts]
        src = flat.clone()
        check(ra, [src[a:b] for a, b in cuts], 0.7, outs=outs)
        mask = torch.ones(60010, dtype=torch.bool, device="cuda")
        for a, b in cuts:
            mask[a + shift:b + shift] = False
        assert (buf[mask] == 3).all()
        rest = torch.ones(60000, dtype=torch.bool, device="cuda")
        for a, b in cuts:
            rest[a:b] = False
        assert torch.equal(src[rest], flat[rest])


@pytest.mark.parametrize("scale", [1e-40, 1e-30, 1e-20, 1e18, 1e30, 2e37])
def test_any_size_of_elements(ra, scale):
    """Squares below and above fp32's range; bf16 reaches as far."""
    check(ra, tensors([5000, 70001, 3], [F, Bf, F], 4, scale), 1.0)
    check(ra, tensors([5000], [F], 5, scale) + tensors([7000], [F], 6), 1.0)


def test_zeros_infinities_and_nans(ra):
    z = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda", dtype=Bf)]
    assert float(ra.grad_clip(z, 1.0)) == 0 and not z[0].any() and not z[1].any()
    x = tensors([5000, 100], [F, Bf], 7)
    x[0][4321] = float("inf")
    a, b = [t.clone() for t in x], [t.clone() for t in x]
    assert float(ra.grad_clip(a, 1.0)) == float("inf")
    assert a[0][4321].isnan() and not a[1].any() and int(a[0].isnan().sum()) == 1
    b[1][3] = float("nan")
    n = ra.grad_clip(b, 1.0)
    assert n.isnan() and b[0].isnan().all() and b[1].isnan().all()
    big = [torch.full((1000,), 3e38, device="cuda")]         # the norm is past fp32, the factor is not
    n = ra.grad_clip(big, 3e38)
    assert float(n) == float("inf") and (big[0] / (3e38 / 1000 ** 0.5) - 1).abs().max() < 1e-5
    ra.ra_sync_status()


def test_same_tensor_twice(ra):
    x = tensors([1000], [F], 8)[0]
    n = ra.grad_norm([x, x])
    assert abs(float(n) - 2 ** 0.5 * float(ra.grad_norm([x]))) < 1e-4
    with pytest.raises(ra.RAError, match="overlap"):
        ra.grad_clip([x, x], 1.0)
    y = torch.empty_like(x)
    with pytest.raises(ra.RAError, match="overlap"):
        ra.grad_clip([x, x.clone()], 1.0, outs=[y, y])


def test_a_tensor_past_32_bits(ra):
    n = 2 ** 31 + 12345
    x = torch.zeros(n, device="cuda", dtype=Bf)
    x[-1], x[2 ** 31 + 5], x[0] = 3.0, 4.0, 12.0
    y = torch.ones_like(x)
    assert float(ra.grad_clip([x], 1.3, outs=[y], eps=0.0)) == 13.0
    assert float(y[-1]) == float(torch.tensor(0.3).to(Bf)) and int((y != 0).sum()) == 3


def test_order_streams_and_graph(ra):
    x = tensors([300000, 1000, 77777], [F, Bf, H], 9)
    outs = [torch.empty_like(t) for t in x]
    want = float(ra.grad_clip(x, 0.1, outs=outs))
    kept = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):  # the same bits each time
        assert float(ra.grad_clip(x, 0.1, outs=outs)) == want
        assert all(torch.equal(a, b) for a, b in zip(outs, kept))
    n = ra.grad_clip(x, 0.1, outs=outs, stream=side)
    side.synchronize()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"] if "address" in b}
    assert owner[n.data_ptr()] == side.cuda_stream and float(n) == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = ra.grad_clip(x, 0.1, outs=outs)
    for t in x:
        t.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(n) - 2 * want) <= 4 * NORM * want
    with pytest.raises(ra.RAError):
        ra.grad_norm([x[0], x[1].cpu()])
    with pytest.raises(ra.RAError):
        ra.grad_norm([x[0][::2]])
    ra.ra_sync_status()
