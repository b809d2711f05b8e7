"""Plain fp64 CPU oracle for the two ends of a training step's backward pass:
the softmax cross entropy of a vocabulary with its gradients, and the
Newton-Schulz orthogonalisation of a weight gradient.

TEST INFRASTRUCTURE ONLY.  Nothing on the CUDA product path imports or calls
this module; it shares no code, header, table or helper with it.  Inputs are
the exact values handed to the GPU, upcast to float64.

Layout: x, dx [T, D] (tokens of all batches flattened), w, dw [V, D], targets
[T] integers; g [rows, cols] or [batch, rows, cols].
"""
import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def xent_fwd(x, w, targets, ignore=-100):
    """loss_t = lse_t - x_t . w_{y_t} with lse_t = ln sum_v e^{x_t . w_v}; a token
    whose target is `ignore` has loss 0.  Returns (loss, lse, logits)."""
    x, w, y = _f64(x), _f64(w), np.asarray(targets)
    z = x @ w.T
    top = z.max(axis=1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    kept = y != ignore
    picked = z[np.arange(len(y)), np.where(kept, y, 0)]
    return np.where(kept, lse - picked, 0.0), lse, z


def xent_bwd(x, w, targets, dloss, ignore=-100):
    """Gradients of sum_t dloss_t loss_t: d_tv = dloss_t (softmax_tv - [v = y_t]),
    dx = d w, dw = d^T x.  Returns (dx, dw, d)."""
    x, w, y = _f64(x), _f64(w), np.asarray(targets)
    _, lse, z = xent_fwd(x, w, y, ignore)
    d = np.exp(z - lse[:, None])
    kept = y != ignore
    d[np.nonzero(kept)[0], y[kept]] -= 1.0
    d *= np.where(kept, _f64(dloss), 0.0)[:, None]
    return d @ w, d.T @ x, d


def newton_schulz(g, coeffs=(3.4445, -4.7750, 2.0315), steps=5, eps=1e-7):
    """X = g / (|g|_F + eps); `steps` times X <- a X + (b A + c A^2) X with A = X X^T
    (taken on the smaller side; (X X^T)^k X = X (X^T X)^k)."""
    g = _f64(g)
    if g.ndim == 3:
        return np.stack([newton_schulz(m, coeffs, steps, eps) for m in g])
    a, b, c = (float(np.float32(v)) for v in coeffs)
    norm = np.sqrt(np.square(g).sum()) + float(np.float32(eps))
    x = g / norm if norm > 0 else np.zeros_like(g)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    return x.T if tall else x


def singular_map(s, coeffs=(3.4445, -4.7750, 2.0315), steps=5):
    """What the iteration does to each singular value: p applied `steps` times,
    p(s) = a s + b s^3 + c s^5."""
    a, b, c = (float(np.float32(v)) for v in coeffs)
    s = _f64(s)
    for _ in range(steps):
        s = s * (a + s * s * (b + c * s * s))
    return s
