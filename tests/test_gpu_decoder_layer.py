"""The operators of a decoder layer together, as a training step and a serving step use them, against
the same layer in fp64 (torch's own products and autograd).

Tolerance of the training step's gradients, in 2-norm: some ten activations and a dozen gradients of
them are rounded to bf16 on the way (each by 2^-8 at most, 0.0017 in the mean square), which add up like
independent errors: 0.0017 sqrt(22) = 0.8%.  3% leaves room for those that a residual or a norm makes
larger."""
import os

import numpy as np
import pytest
import torch

import oracle

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu

N, DM, H, HK, D, DH, P, BE, NE, V, EPS = 512, 256, 4, 2, 64, 512, 4, 1, 301, 1000, 1e-5
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ra():
    import blockwise_exact_attention_ra_gb300 as ra
    yield ra
    ra.ra_sync_status()


def parameters():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def w(*s):
        return (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).to(BF)

    p = dict(wq=w(H * D, DM), wk=w(HK * D, DM), wv=w(HK * D, DM), wo=w(DM, H * D), cq=w(H * D, DM), ck=w(HK * D, DM),
             cv=w(HK * D, DM), co=w(DM, H * D), w1=w(DH, DM), w2=w(DM, DH), vocab=w(V, DM))
    for n in ("qn", "kn", "cn"):
        p[n] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(BF)
    x = torch.randn(N, DM, generator=g, device="cuda").to(BF)
    enc = torch.randn(BE * NE, DM, generator=g, device="cuda").to(BF)
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    y[::7] = -100
    return p, x, enc, y, torch.tensor([257], dtype=torch.int32, device="cuda")


def reference(p, x, enc, y, n_keys, freq):
    """Loss and gradients in fp64; rows are in striped order."""
    p = {k: t.double().requires_grad_() for k, t in p.items()}
    x = x.double().requires_grad_()
    pos = torch.tensor(oracle.rows_to_positions(N, P, True), device="cuda")

    def norm(t, w):
        return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w

    def rotate(t):
        a = pos[:, None].double() * freq
        c, s = a.cos()[:, None], a.sin()[:, None]
        u, v = t[..., :D // 2], t[..., D // 2:]
        return torch.cat((u * c - v * s, u * s + v * c), -1)

    def attend(q, k, v, mask):
        k, v = (t.repeat_interleave(H // HK, dim=1) for t in (k, v))
        z = torch.einsum("nhd,mhd->hnm", q, k) * D ** -0.5
        return torch.einsum("hnm,mhd->nhd", z.masked_fill(~mask, -torch.inf).softmax(-1), v).reshape(N, H * D)

    q, k, v = ((x @ p[n].T).view(N, -1, D) for n in ("wq", "wk", "wv"))
    h = x + attend(rotate(norm(q, p["qn"])), rotate(norm(k, p["kn"])), v, pos[None, :] <= pos[:, None]) @ p["wo"].T
    ck, cv = ((enc.double() @ p[n].T).view(NE, HK, D) for n in ("ck", "cv"))
    cq = norm((h @ p["cq"].T).view(N, H, D), p["cn"])
    h = h + attend(cq, ck, cv, torch.arange(NE, device="cuda")[None, :] < n_keys) @ p["co"].T
    h = h + torch.nn.functional.gelu(h @ p["w1"].T) @ p["w2"].T
    loss = torch.nn.functional.cross_entropy(h @ p["vocab"].T, y, ignore_index=-100, reduction="sum") / N
    loss.backward()
    return float(loss.detach()), dict({k: t.grad for k, t in p.items()}, x=x.grad)


def step(ra, p, x, enc, y, kv_len, freq):
    """The same with the library's operators; returns the loss and the gradients."""
    g = {}
    ring = dict(P=P, causal=True, striped=True)
    rows = dict(eps=EPS, P=P, striped=True)
    q, k, v = ((x @ p[n].T).view(1, N, -1, D) for n in ("wq", "wk", "wv"))
    qr, kr = ra.norm_rotary_fwd(q, k, p["qn"], p["kn"], freq, **rows)
    o, lse = ra.ring_attention_fwd(qr, kr, v, o_dtype=BF, **ring)
    h1 = x + o.view(N, -1) @ p["wo"].T
    ck, cv = ((enc @ p[n].T).view(BE, NE, HK, D) for n in ("ck", "cv"))
    cq = (h1 @ p["cq"].T).view(1, N, H, D)
    cqn, _ = ra.norm_rotary_fwd(cq, None, p["cn"], None, None, eps=EPS)
    c, clse = ra.cross_attention_fwd(cqn, ck, cv, kv_len, o_dtype=BF)
    h2 = h1 + c.view(N, -1) @ p["co"].T
    h3 = h2 + ra.ffn_fwd(h2, p["w1"], p["w2"], 256)
    loss, zl = ra.xent_fwd(h3, p["vocab"], y)
    weight = torch.full((N,), 1.0 / N, device="cuda")
    dh, g["vocab"] = ra.xent_bwd(h3, p["vocab"], y, zl, weight, dx_dtype=BF)
    dx2, g["w1"], g["w2"] = ra.ffn_bwd(h2, p["w1"], p["w2"], dh, 256)
    dh = (dh + dx2).to(BF)
    g["co"] = dh.T.float() @ c.view(N, -1).float()
    dcqn, dck, dcv = ra.cross_attention_bwd(cqn, ck, cv, c, clse, (dh @ p["co"]).view(1, N, H, D), kv_len, grad_dtype=BF)
    g["ck"], g["cv"] = (t.view(NE, -1).T.float() @ enc.float() for t in (dck, dcv))
    dcq, _, g["cn"], _ = ra.norm_rotary_bwd(cq, None, dcqn, None, p["cn"], None, None, eps=EPS)
    g["cq"] = dcq.view(N, -1).T.float() @ h1.float()
    dh = (dh.float() + (dcq.view(N, -1) @ p["cq"]).float()).to(BF)
    g["wo"] = dh.T.float() @ o.view(N, -1).float()
    dqr, dkr, dv = ra.ring_attention_bwd(qr, kr, v, o, lse, (dh @ p["wo"]).view(1, N, H, D), **ring)  # fp32
    dq, dk, g["qn"], g["kn"] = ra.norm_rotary_bwd(q, k, dqr, dkr, p["qn"], p["kn"], freq, grad_dtype=BF, **rows)
    dx = dh.float()
    for n, t in (("wq", dq), ("wk", dk), ("wv", dv.to(BF))):
        t = t.reshape(N, -1)
        g[n] = t.T.float() @ x.float()
        dx = dx + (t @ p[n]).float()
    g["x"] = dx
    return float(loss.sum()) / N, g


def test_training_step(ra):
    p, x, enc, y, kv_len = parameters()
    freq = ra.rotary_frequencies(D, 10000.0, 2.0, "parts", trained=256)
    want_loss, want = reference(p, x, enc, y, int(kv_len), freq)
    loss, g = step(ra, p, x, enc, y, kv_len, freq)
    ra.ra_sync_status()
    assert abs(loss - want_loss) < 3e-3 * want_loss
    for n, t in want.items():
        off = float((g[n].double() - t).norm() / t.norm())
        assert off < 3e-2, (n, off)
    # the update: clipped by the common norm, then orthogonalised
    names = sorted(n for n in g if n != "x")
    grads = [g[n].contiguous() for n in names]
    norm = float(torch.stack([t.double().square().sum() for t in grads]).sum().sqrt())
    max_norm = norm / 3
    outs = [torch.empty(t.shape, dtype=BF if t.dim() == 2 else t.dtype, device="cuda") for t in grads]
    got = ra.grad_clip(grads, max_norm, outs=outs)
    assert abs(float(got) - norm) < 2e-6 * norm
    for t, o in zip(grads, outs):
        c = t.double() * min(1.0, float(np.float32(max_norm)) / (norm + 1e-6))
        assert ((o.double() - c).abs() <= c.abs() * (torch.finfo(o.dtype).eps / 2 * 1.01 + 2e-6) + 1e-38).all()
    w1 = outs[names.index("w1")]
    update = ra.newton_schulz(w1, out_dtype=torch.float32)
    assert (update.double().cpu() - torch.tensor(oracle.newton_schulz(w1.double().cpu().numpy()))).norm() < 8e-3 * update.double().norm().cpu()
    ra.ra_sync_status()


def test_serving_step_from_a_graph(ra):
    """One token a call: its query normed and rotated at its own position, attention to an encoder's
    states; captured once and replayed for the tokens that follow."""
    B, Ne = 3, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def rand(*s):
        return torch.randn(s, generator=g, device="cuda").to(BF)

    k, v, w = rand(B, Ne, HK, D), rand(B, Ne, HK, D), rand(D)
    kv_len = torch.tensor([700, 1, 333], dtype=torch.int32, device="cuda")
    freq = ra.rotary_frequencies(D)
    q, pos = rand(B, 1, H, D), torch.zeros(B, 1, dtype=torch.int64, device="cuda")

    def token():
        qr, _ = ra.norm_rotary_fwd(q, None, w, None, freq, positions=pos)
        return qr, *ra.cross_attention_fwd(qr, k, v, kv_len)

    token()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    for i in range(3):
        q.copy_(rand(B, 1, H, D))
        pos.copy_(torch.tensor([[1000 * i], [7], [2 ** 20 + i]], device="cuda"))
        graph.replay()
        want = token()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        o, lse = oracle.cross_attention(want[0].double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(),
                                        D ** -0.5, kv_len.tolist())
        assert np.abs(want[1].double().cpu().numpy() - o).max() < 2.0 ** -14 * float(v.abs().max())
        assert np.abs(want[2].double().cpu().numpy() - lse).max() < 1e-4
    ra.ra_sync_status()
