"""Pins of the fp64 oracle of rotary positions, norms of heads, cross attention and
clipping: closed forms, invariants and differences."""
import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_by_hand(interleaved):
    x = np.arange(1.0, 7.0).reshape(1, 1, 1, 6)
    out = oracle.rotary(x, [3], [0.5, 0.25], interleaved, 2.0)[0, 0, 0]
    pairs = [(0, 1), (2, 3)] if interleaved else [(0, 2), (1, 3)]
    for (i, j), f in zip(pairs, (0.5, 0.25)):
        c, s = np.cos(3 * f), np.sin(3 * f)
        assert np.allclose(out[[i, j]], [2 * ((i + 1) * c - (j + 1) * s), 2 * ((i + 1) * s + (j + 1) * c)])
    assert (out[4:] == [5, 6]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_products_depend_on_distances(interleaved):
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 1, 8))
    f = 10.0 ** -np.arange(4)

    def dot(p, r):
        return float((oracle.rotary(q, [p], f, interleaved) * oracle.rotary(k, [r], f, interleaved)).sum())

    assert dot(7, 3) == pytest.approx(dot(104, 100)) and dot(7, 3) != pytest.approx(dot(8, 3))


def test_rotary_transpose_is_the_gradient():
    rng = np.random.default_rng(1)
    x, g = rng.normal(size=(2, 2, 3, 2, 10))
    p, f = rng.integers(0, 99, (2, 3)), rng.uniform(0, 1, 3)
    lhs = (g * oracle.rotary(x, p, f, False, 1.3)).sum()
    assert lhs == pytest.approx((x * oracle.rotary(g, p, f, False, 1.3, transpose=True)).sum())


def test_striped_positions():
    assert oracle.rows_to_positions(6, 3, True).tolist() == [0, 3, 1, 4, 2, 5]
    assert oracle.rows_to_positions(3, pos_off=5).tolist() == [5, 6, 7]


def test_head_norm_gradients_are_differences():
    rng = np.random.default_rng(2)
    x, dn, w = rng.normal(size=(1, 2, 2, 5)), rng.normal(size=(1, 2, 2, 5)), rng.normal(size=5)

    def f(x, w):
        return (dn * oracle.head_norm(x, w, 1e-3)[0]).sum()

    dx, dw = oracle.head_norm_bwd(x, dn, w, 1e-3)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert (f(x + e, w) - f(x - e, w)) / (2 * h) == pytest.approx(dx[at], abs=1e-7)
    for c in range(5):
        e = np.zeros(5)
        e[c] = h
        assert (f(x, w + e) - f(x, w - e)) / (2 * h) == pytest.approx(dw[c], abs=1e-7)


def test_cross_attention_by_hand_and_differences():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(2, 3, 4, 3)), rng.normal(size=(2, 5, 2, 3)), rng.normal(size=(2, 5, 2, 3))
    do = rng.normal(size=q.shape)
    lens = [5, 2]
    o, lse, dq, dk, dv = oracle.cross_attention(q, k, v, 0.7, lens, do)
    z = 0.7 * k[1, :2, 1] @ q[1, 2, 3]
    assert o[1, 2, 3] == pytest.approx((np.exp(z) / np.exp(z).sum()) @ v[1, :2, 1])
    assert lse[1, 3, 2] == pytest.approx(np.log(np.exp(z).sum()))
    assert (dk[1, 2:] == 0).all() and (dv[1, 2:] == 0).all()
    h = 1e-6
    for name, t, g in (("q", q, dq), ("k", k, dk), ("v", v, dv)):
        for at in ((0, 1, 0, 2), (1, 1, 1, 0)):
            e = np.zeros_like(t)
            e[at] = h
            up, down = ((do * oracle.cross_attention(*(x + s * e if n == name else x for n, x in
                         (("q", q), ("k", k), ("v", v))), 0.7, lens)[0]).sum() for s in (1, -1))
            assert (up - down) / (2 * h) == pytest.approx(g[at], abs=1e-7)


def test_cross_attention_without_keys_and_as_self_attention():
    rng = np.random.default_rng(4)
    q, k, v, do = rng.normal(size=(4, 1, 6, 2, 4))
    o, lse, dq, dk, dv = oracle.cross_attention(q, k, v, 0.5, [0], do)
    assert (o == 0).all() and (lse == -np.inf).all() and not dq.any() and not dk.any() and not dv.any()
    got = oracle.cross_attention(q, k, v, 0.5, None, do)
    rq, rk, rv, ro, rl, _ = oracle.attention_bwd(q, k, v, do, False, 0.5)
    for a, b in zip(got, (ro, rl, rq, rk, rv)):
        assert np.allclose(a, b)


def test_clip_factor():
    n = oracle.global_norm([np.array([3.0]), np.array([[0.0, 4.0]])])
    assert n == 5.0 and oracle.clip_factor(n, 10.0) == 1.0
    assert oracle.clip_factor(n, 1.0, 0.0) == pytest.approx(0.2)
