"""Plain fp64 CPU oracle for the operators of a decoder layer that stand beside its
self attention: rotary positions, the norms of queries and keys for each head,
cross attention to keys of another length, and clipping by the global norm.

TEST INFRASTRUCTURE ONLY.  Nothing on the CUDA product path imports or calls this
module; it shares no code, header, table or helper with it.  Inputs are the exact
values handed to the GPU, upcast to float64.

Layout: q, k, v [B, N, H, d]; positions [N] or [B, N] integers; freq [rot / 2].
"""
import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def rotary(x, positions, freq, interleaved=False, amplitude=1.0, transpose=False):
    """Pairs (i, i + n) or (2i, 2i + 1) of the first 2 n columns as complex numbers, times
    amplitude e^{i p freq} (its conjugate: the transpose)."""
    x, freq = _f64(x), _f64(freq)
    n = len(freq)
    p = np.asarray(positions)
    if p.ndim == 1:
        p = p[None]
    # the angle modulo a turn, exactly enough for any 64-bit position
    a = p.astype(np.longdouble)[..., None] * freq.astype(np.longdouble)
    turn = amplitude * np.exp((-1j if transpose else 1j) * a.astype(np.float64))[:, :, None]
    out = x.copy()
    if interleaved:
        z = (x[..., 0:2 * n:2] + 1j * x[..., 1:2 * n:2]) * turn
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = (x[..., :n] + 1j * x[..., n:2 * n]) * turn
        out[..., :n], out[..., n:2 * n] = z.real, z.imag
    return out


def rows_to_positions(N, P=1, striped=False, pos_off=0):
    """Positions of N rows: as they are, or host i's row l at l P + i."""
    row = np.arange(N)
    if striped:
        S = N // P
        row = row % S * P + row // S
    return row + pos_off


def head_norm(x, w=None, eps=1e-6):
    x = _f64(x)
    r = 1.0 / np.sqrt(np.square(x).mean(axis=-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else _f64(w)), r


def head_norm_bwd(x, dn, w=None, eps=1e-6):
    """Gradients of sum(dn * head_norm(x, w)): dx, dw."""
    x, dn = _f64(x), _f64(dn)
    w = np.ones(x.shape[-1]) if w is None else _f64(w)
    n, r = head_norm(x, None, eps)
    u = dn * w
    return r * (u - n * (u * n).mean(axis=-1, keepdims=True)), (dn * n).sum(axis=(0, 1, 2))


def cross_attention(q, k, v, scale, lens=None, do=None):
    """softmax(scale q k^T) v over the first lens[b] keys (all by default), one batch entry
    and head at a time.  Returns o, lse, and with `do` also dq, dk, dv.  No key: o = 0,
    lse = -inf, no gradient."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Nq, Hq, d = q.shape
    Nkv, Hkv = k.shape[1:3]
    o, lse = np.zeros_like(q), np.full((B, Hq, Nq), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        n = Nkv if lens is None else min(max(int(lens[b]), 0), Nkv)
        if n == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            K, V = k[b, :n, g], v[b, :n, g]
            z = scale * q[b, :, h] @ K.T
            top = z.max(axis=1, keepdims=True)
            p = np.exp(z - top)
            total = p.sum(axis=1, keepdims=True)
            p /= total
            o[b, :, h] = p @ V
            lse[b, h] = (top + np.log(total))[:, 0]
            if do is not None:
                g_o = _f64(do)[b, :, h]
                dp = g_o @ V.T
                ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
                dv[b, :n, g] += p.T @ g_o
                dq[b, :, h] = scale * ds @ K
                dk[b, :n, g] += scale * ds.T @ q[b, :, h]
    return (o, lse) if do is None else (o, lse, dq, dk, dv)


def global_norm(tensors):
    return float(np.sqrt(sum(np.square(_f64(t)).sum() for t in tensors)))


def clip_factor(norm, max_norm, eps=1e-6):
    return min(1.0, max_norm / (norm + eps))
