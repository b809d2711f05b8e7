"""Angles of far positions at frequencies of any size, against integers of as many bits as they take.

A turned column is x C + x' S in fp32: 5e-7 (|x| + |x'|) for sine, cosine, products and sum (fp32
rows), and 2 pi 2^-64 |p| of a radian times |x| + |x'| for the angle."""
import math
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests._parity import f64

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


@pytest.mark.parametrize("frequencies", [(1.0, 0.95, 0.83, 0.5001), (2.5, 6.2, 7.3, 100.0), (1e-3, 1e-7, 3e-19, 0.0),
                                         (-0.9, -1e-30, -1234.5, -math.pi), (1e6, 1e9, math.pi, 2 * math.pi)])
def test_far_positions(ra, frequencies):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    p = [0, 1, -1, 2 ** 24 + 1, -2 ** 31, 2 ** 40 + 12345, 3 ** 28, -5 ** 19, 2 ** 46 + 1]
    x = torch.randn((1, len(p), 2, 8), generator=g, device="cuda")
    freq = torch.tensor(frequencies, dtype=torch.float64, device="cuda")
    y, _ = ra.rotary_fwd(x, None, freq, positions=torch.tensor(p, device="cuda"))
    back, _ = ra.rotary_bwd(y, None, freq, positions=torch.tensor(p, device="cuda"))
    ra.ra_sync_status()
    X, want, lim = f64(x), np.empty(x.shape), np.empty(x.shape)
    for n, pos in enumerate(p):
        for i, f in enumerate(frequencies):
            turns = Fraction(pos) * Fraction(f) / (2 * PI) % 1
            a = 2 * math.pi * float(turns)
            u, v = X[0, n, :, i], X[0, n, :, i + 4]
            want[0, n, :, i], want[0, n, :, i + 4] = u * math.cos(a) - v * math.sin(a), u * math.sin(a) + v * math.cos(a)
            lim[0, n, :, i] = lim[0, n, :, i + 4] = (np.abs(u) + np.abs(v)) * (5e-7 + 2 * math.pi * abs(pos) * 2.0 ** -64)
    err = np.abs(f64(y) - want)
    assert (err <= lim).all(), (err / lim).max(axis=(0, 2))
    size = (X[..., :4] ** 2 + X[..., 4:] ** 2) ** 0.5
    assert (np.abs(f64(back) - X) <= 2e-6 * np.concatenate((size, size), axis=-1)).all()
