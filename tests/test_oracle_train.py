"""Pins for the fp64 oracle of the cross entropy and the Newton-Schulz update,
independent of its own formulas: closed forms, invariants, finite differences,
torch's autograd on tiny inputs, and planted mistakes that these pins catch."""
import numpy as np
import pytest

import oracle

RNG = np.random.default_rng(20260601)


def _case(T=6, D=5, V=9, ignored=(2,)):
    x, w = RNG.standard_normal((T, D)), RNG.standard_normal((V, D))
    y = RNG.integers(0, V, T)
    y[list(ignored)] = -100
    return x, w, y, RNG.standard_normal(T)


def test_equal_logits_give_log_of_the_vocabulary():
    loss, lse, _ = oracle.xent_fwd(np.zeros((3, 4)), RNG.standard_normal((7, 4)), [0, 6, 3])
    np.testing.assert_allclose(loss, np.log(7.0), atol=1e-15)
    np.testing.assert_allclose(lse, np.log(7.0), atol=1e-15)


def test_two_entries_are_a_sigmoid():
    x, w = np.array([[1.0]]), np.array([[2.0], [-1.0]])
    loss, _, _ = oracle.xent_fwd(x, w, [1])
    np.testing.assert_allclose(loss, np.log1p(np.exp(3.0)), rtol=1e-15)


def test_a_common_shift_changes_lse_and_not_loss():
    x, w, y, _ = _case(ignored=())
    x1, w1 = np.c_[x, np.ones(len(x))], np.c_[w, np.full(len(w), 0.0)]
    w2 = np.c_[w, np.full(len(w), 2.5)]
    (la, ea, _), (lb, eb, _) = oracle.xent_fwd(x1, w1, y), oracle.xent_fwd(x1, w2, y)
    np.testing.assert_allclose(lb, la, atol=1e-13)
    np.testing.assert_allclose(eb, ea + 2.5, atol=1e-13)


def test_gradients_of_the_logits_sum_to_zero_and_ignored_rows_vanish():
    x, w, y, g = _case()
    dx, _, d = oracle.xent_bwd(x, w, y, g)
    np.testing.assert_allclose(d.sum(axis=1), 0.0, atol=1e-14)
    assert not d[2].any() and not dx[2].any()


def test_gradients_by_finite_differences():
    x, w, y, g = _case()
    dx, dw, _ = oracle.xent_bwd(x, w, y, g)
    eps = 1e-6
    for arr, grad, which in ((x, dx, 0), (w, dw, 1)):
        fd = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            p, m = arr.copy(), arr.copy()
            p[i] += eps
            m[i] -= eps
            lp = oracle.xent_fwd(*((p, w) if which == 0 else (x, p)), y)[0] @ g
            lm = oracle.xent_fwd(*((m, w) if which == 0 else (x, m)), y)[0] @ g
            fd[i] = (lp - lm) / (2 * eps)
        np.testing.assert_allclose(grad, fd, rtol=1e-6, atol=1e-8)


def test_matches_torch_with_autograd():
    torch = pytest.importorskip("torch")
    x, w, y, g = _case()
    tx, tw = (torch.tensor(a, dtype=torch.float64, requires_grad=True) for a in (x, w))
    loss = torch.nn.functional.cross_entropy(tx @ tw.T, torch.tensor(y), reduction="none", ignore_index=-100)
    loss.backward(torch.tensor(g))
    dx, dw, _ = oracle.xent_bwd(x, w, y, g)
    np.testing.assert_allclose(oracle.xent_fwd(x, w, y)[0], loss.detach().numpy(), atol=1e-13)
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-13)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (6, 6), (1, 5), (5, 1)])
def test_newton_schulz_acts_on_the_singular_values(shape):
    g = RNG.standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    want = (u * oracle.singular_map(s / (np.linalg.norm(g) + 1e-7))) @ vt
    np.testing.assert_allclose(oracle.newton_schulz(g), want, atol=1e-12)


def test_newton_schulz_brings_singular_values_near_one():
    s = oracle.singular_map(np.geomspace(3e-3, 1.0, 200))
    assert s.min() > 0.5 and s.max() < 1.3


def test_newton_schulz_invariants():
    g = RNG.standard_normal((5, 8))
    x = oracle.newton_schulz(g, eps=0.0)
    np.testing.assert_allclose(oracle.newton_schulz(37.0 * g, eps=0.0), x, atol=1e-13)   # scale
    np.testing.assert_allclose(oracle.newton_schulz(g.T, eps=0.0), x.T, atol=1e-13)      # transpose
    q, _ = np.linalg.qr(RNG.standard_normal((5, 5)))
    np.testing.assert_allclose(oracle.newton_schulz(q @ g, eps=0.0), q @ x, atol=1e-12)  # rotation
    assert not oracle.newton_schulz(np.zeros((3, 4))).any()
    both = oracle.newton_schulz(np.stack([g, 2 * g]), eps=0.0)
    np.testing.assert_allclose(both[0], both[1], atol=1e-13)


def test_planted_mistakes_are_caught():
    x, w, y, g = _case(ignored=())
    dx, dw, d = oracle.xent_bwd(x, w, y, g)
    soft = d + g[:, None] * (np.arange(len(w))[None] == y[:, None])
    assert np.abs(soft @ w - dx).max() > 1e-3           # the one-hot term left out
    assert np.abs((d / g[:, None]).T @ x - dw).max() > 1e-3   # the token's weight left out
    m = RNG.standard_normal((5, 8))
    a = m / np.linalg.norm(m, 2)                         # spectral norm in place of Frobenius
    assert np.abs(oracle.newton_schulz(m, eps=0.0) - (a * 3.4445)).max() > 1e-3
