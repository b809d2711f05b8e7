"""Gradients whose norm is far below eps: X = G / (|G| + eps) is then tiny and grows by the
polynomial's slope at zero, 3.4445, with every step.  The result is as exact as for any other
gradient: the operands' errors are those of fp16 values of ordinary size, 2^-11 of each product, which
for a tiny X change only what the products add to a X; the two terms that hold X are exact to 2^-21 of
its largest entries, and half a step of their lowest bit, 2^-25, next to entries that are held times
the square root of the matrix's size, so between 2^-3 and 1 in the mean: 2^-22 per step.  Over 5 steps
and with every step's error passed on in proportion that is below 1e-5; where the norm has grown to
1e-2 and more the products count, and the bound is that of ordinary gradients, 2e-3."""
import os

import numpy as np
import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

import oracle  # noqa: E402
from tests._parity import f64  # noqa: E402

pytestmark = pytest.mark.gpu


def rel(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    assert torch.cuda.is_available()
    return ra


def unit(rows, cols, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g = torch.randn(rows, cols, generator=gen, device="cuda")
    return g / g.norm()


@pytest.mark.parametrize("rows,cols", [(100, 300), (200, 300), (300, 200), (140, 4500), (700, 1030)])
@pytest.mark.parametrize("ratio", [0.3, 1e-2, 1e-4, 1e-5, 1e-7, 1e-9, 1e-15, 1e-25])
def test_norms_far_below_eps(ra, rows, cols, ratio):
    g = unit(rows, cols, 81) * (ratio * 1e-3)
    o = ra.newton_schulz(g, eps=1e-3)
    ra.ra_sync_status()
    want = oracle.newton_schulz(f64(g), eps=1e-3)
    assert rel(f64(o), want) <= (2e-3 if ratio > 1e-5 else 1e-5)


@pytest.mark.parametrize("rows,cols", [(100, 300), (200, 300), (300, 200)])
@pytest.mark.parametrize("steps,ratio", [(1, 1e-6), (12, 1e-6), (20, 1e-9), (24, 1e-12)])
def test_steps_that_bring_them_to_size(ra, rows, cols, steps, ratio):
    """a^12 = 2.8e6, a^20 = 5.5e10, a^24 = 7.7e12: X grows from nothing to singular values near one."""
    g = unit(rows, cols, 82) * ratio
    o = ra.newton_schulz(g, eps=1.0, steps=steps)
    ra.ra_sync_status()
    want = oracle.newton_schulz(f64(g), eps=1.0, steps=steps)
    if steps > 1:
        assert np.linalg.norm(want) > 1.0
    assert rel(f64(o), want) <= (2e-3 if steps > 1 else 1e-5)


def test_a_batch_of_all_sizes(ra):
    """Each matrix of a batch has its own power of two, and the same result as by itself; a zero one
    gives zero."""
    ratios = [1.0, 1e-3, 0.0, 1e-6, 1e-12, 0.25, 1e-20]
    g = torch.stack([unit(150, 260, 83 + i) * (r * 1e-2) for i, r in enumerate(ratios)])
    o = ra.newton_schulz(g, eps=1e-2)
    for i, r in enumerate(ratios):
        assert torch.equal(o[i], ra.newton_schulz(g[i], eps=1e-2)), i
        if r == 0.0:
            assert not o[i].any()
        else:
            assert rel(f64(o[i]), oracle.newton_schulz(f64(g[i]), eps=1e-2)) <= 2e-3
    ra.ra_sync_status()


@pytest.mark.parametrize("rows,cols", [(200, 300), (300, 200)])
def test_ordinary_norms_keep_their_results(ra, rows, cols):
    """No power of two is taken where the norm is eps or more: the same bits as with eps of 0 where eps
    does not change the quotient."""
    g = unit(rows, cols, 90) * 4.0
    assert torch.equal(ra.newton_schulz(g, eps=0.0), ra.newton_schulz(g, eps=1e-30))
    ra.ra_sync_status()
