"""The gradient of tokens that the model is sure of.

Token t leans so far towards its target y that its loss l = ln(1 + R), R the other
entries' weight, is 1e-3 to 1e-4, and the target's element of the logits' gradient is
-g (1 - e^-l) = -g l, nearly.  The products that make up its logit are all positive, so
that the tensor core's sums, which round towards zero, are off to one side by as much as
they can be.  What has to hold: the backward's logit is the forward's, so that error
leaves z_y - lse; what remains of it is, absolutely,
  e_a = |z| 2^-23 (the exponent's argument, two roundings) + 2^-21 (the exponential's and
        the sums' relative errors, next to a largest term of 1) + 2^-23 |lse| (the
        logarithm and lse's own rounding, half a step of at most 2^-23 |lse|),
and, relative to R, twice the logits' error e_z.  A logit is the sum, in fp32, of pieces
of at most 768 products, 48 steps of 16 that each lose at most 2^-23 of the partial sum:
  e_z = (48 + D / 768) 2^-23 s, s = max_v sum_k |x_k w_vk|.
(Sums over the whole of D lose D / 16 steps: at 16384 products 1e-4 of a logit of 14.)
An element of d is then within |g| p (e_z + e_lse), the target's within |g| p (e_a + 2 e_z l),
and u |d|, u = 2^-8 (bf16) or 2^-11 (fp16), u^2 |d| + 2^-22 |d| for up to 64 tokens; in fp16 the
subnormals add g_max 2^-38.  dx and dw: the sums of these errors times the other factor, and
K 2^-23 of the absolute products."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("T,D,V", [(1, 8192, 512), (16, 4096, 512), (17, 2048, 300), (17, 16384, 512), (64, 16384, 512),
                                   (65, 16384, 512), (300, 16384, 1000), (300, 2048, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients_of_sure_tokens(T, D, V, dtype):
    import blockwise_exact_attention_ra_gb300 as ra
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + D)
    w = torch.randn(V, D, generator=gen, device="cuda").to(dtype)
    y = torch.randperm(V, generator=gen, device="cuda")[:T]
    lean = 14.0 + 1.5 * torch.rand(T, 1, generator=gen, device="cuda")
    x = (lean * w[y].float() / w[y].float().square().sum(1, keepdim=True)).to(dtype)
    g = 0.5 + torch.rand(T, generator=gen, device="cuda")
    loss, lse = ra.xent_fwd(x, w, y)
    dx, dw = ra.xent_bwd(x, w, y, lse, g)
    ra.ra_sync_status()

    X, W, G = x.double(), w.double(), g.double()
    z = X @ W.T
    rows = torch.arange(T, device="cuda")
    others = z.clone()
    others[rows, y] = float("-inf")
    ref = torch.log1p(torch.exp(others - z[rows, y][:, None]).sum(1))
    assert 1e-5 < float(ref.min()) and float(ref.max()) < 2e-3
    e_z = (48 + D / 768) * 2.0 ** -23 * (X.abs() @ W.abs().T).amax(1)
    top = z[rows, y].abs()
    e_a = top * 2.0 ** -23 + 2.0 ** -21 + 2.0 ** -23 * (top + ref)
    worst = float(((loss.double() - ref).abs() - (e_a + 2 * e_z * ref)).max())
    assert worst <= 0.0, f"loss: past its bound by {worst:.3e}"

    p = torch.softmax(z, 1)
    d = p * G[:, None]
    d[rows, y] = -torch.expm1(-ref) * G
    e_d = G[:, None] * p * (2 * e_z + e_a)[:, None]
    e_d[rows, y] = G * (e_a + 2 * e_z * ref)
    u = U[dtype]
    e_d += (1.01 * (u * u if T <= 64 else u) + 2.0 ** -22) * d.abs()
    if dtype == torch.float16:
        e_d += float(G.max()) * 2.0 ** -38
    d[rows, y] *= -1
    for name, got, want, bound in (
            ("dx", dx, d @ W, e_d @ W.abs() + 2 * V * 2.0 ** -23 * (d.abs() @ W.abs())),
            ("dw", dw, d.T @ X, e_d.T @ X.abs() + 2 * T * 2.0 ** -23 * (d.abs().T @ X.abs()))):
        off = (got.double() - want).abs()
        worst = float((off - bound - 2.0 ** -24 * want.abs()).max())
        assert worst <= 0.0, f"{name}: past its bound by {worst:.3e} (norm {float(off.norm() / want.norm()):.2e})"
