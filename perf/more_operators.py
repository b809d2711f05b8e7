"""Cases for the operators of a decoder layer that stand beside its self attention
and feed-forward layer: rotary positions of queries and keys, the norms of queries
and keys for each head with that rotation in the same pass, cross attention to an
encoder's states of another length, and the global gradient norm with clipping
that comes before the update.

A case is one call as a user's program makes it (`op`):
  "rotary"      queries and keys rotated by their positions
  "rotary_grad" the gradient of that
  "norm"        queries and keys normed for each head and rotated
  "norm_step"   that with its gradients, as a training step calls it
  "cross"       cross attention alone (serving)
  "cross_step"  cross attention with its gradients
  "clip"        gradients of many tensors clipped by their common norm
With ``own`` false, ``run`` computes the plain form in 32 bits (angles in 64, where
32 bits lose those of far positions) from elementary torch operations; with ``own``
true it calls the framework's operators."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NORM_EPS = 1e-6
CLIP_EPS = 1e-6


def listed():
    return [
        # decoding: one new token of each of many sequences, at positions of their own, far ones among them
        dict(name="rotary decode", op="rotary", B=64, N=1, Hq=16, Hkv=16, d=128, rot=128, dtype="bf16",
             interleaved=False, positions="far", P=1, scaled=1.0),
        # the queries and keys of a sequence far longer than the trained ones (frequencies scaled), in the ring's
        # striped order, half of each head rotated
        dict(name="rotary long striped", op="rotary", B=1, N=131072, Hq=16, Hkv=16, d=128, rot=64, dtype="bf16",
             interleaved=True, positions="striped", P=32, scaled=8.0),
        # what the attention's backward pass returns in fp32, odd sizes and a part of the head that no vector divides
        dict(name="rotary gradient ragged", op="rotary_grad", B=3, N=1777, Hq=12, Hkv=3, d=80, rot=20, dtype="fp32",
             interleaved=False, positions="given", P=1, scaled=1.0),
        # decoding with normed queries and keys
        dict(name="norm decode", op="norm", B=32, N=1, Hq=32, Hkv=8, d=128, rot=128, dtype="bf16",
             interleaved=False, positions="far", P=1, scaled=4.0),
        # one training step of a long sequence with grouped heads
        dict(name="norm step long", op="norm_step", B=1, N=131072, Hq=16, Hkv=4, d=128, rot=128, dtype="bf16",
             interleaved=False, positions="rows", P=1, scaled=1.0),
        # a training step of odd sizes with small heads
        dict(name="norm step ragged fp16", op="norm_step", B=3, N=1001, Hq=8, Hkv=8, d=64, rot=32, dtype="fp16",
             interleaved=True, positions="given", P=1, scaled=1.0),
        # decoding against encoders of several lengths, grouped heads
        dict(name="cross decode", op="cross", B=16, Nq=1, Nkv=4096, Hq=32, Hkv=8, d=128, dtype="bf16", ragged=True),
        # a few drafted tokens against one very long document
        dict(name="cross few long", op="cross", B=1, Nq=5, Nkv=131072, Hq=16, Hkv=4, d=128, dtype="fp16", ragged=False),
        # a training step of a padded batch of odd sizes, one of its encoders empty
        dict(name="cross step ragged fp16", op="cross_step", B=4, Nq=333, Nkv=1500, Hq=8, Hkv=2, d=64, dtype="fp16",
             ragged=True),
        # a training step against a long encoder
        dict(name="cross step long", op="cross_step", B=2, Nq=8192, Nkv=8192, Hq=16, Hkv=16, d=128, dtype="bf16",
             ragged=False),
        # the gradients of a small layer
        dict(name="clip small", op="clip", tensors=6, elements=100003, dtype="fp32"),
        # the gradients of a stack of layers: large matrices and many small vectors
        dict(name="clip stack of layers", op="clip", tensors=300, elements=2 ** 29, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "norm", "norm_step", "cross", "cross", "cross_step", "clip"])
    if op == "clip":
        tensors = _log_int(rng, 1, 400)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return dict(op=op, tensors=tensors, elements=_log_int(rng, 40 * tensors, 2 ** (28 if dtype == "fp32" else 29)),
                    dtype=dtype)
    if op in ("cross", "cross_step"):
        while True:
            hkv, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4, 8])
            c = dict(op=op, B=_log_int(rng, 1, 32), Nq=_log_int(rng, 1, 8192), Nkv=_log_int(rng, 1, 131072),
                     Hq=hkv * group, Hkv=hkv, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "fp16"]),
                     ragged=rng.random() < 0.5)
            if op == "cross" and rng.random() < 0.4:
                c["Nq"] = rng.randint(1, 8)
            if c["Hq"] <= 32 and c["B"] * c["Hq"] * c["Nq"] * c["Nkv"] <= 2 ** 31 and \
                    c["B"] * c["Hkv"] * c["Nkv"] * c["d"] <= 2 ** 28:
                return c
    while True:
        hkv, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4, 7])
        d = rng.choice([32, 64, 80, 96, 128, 256])
        c = dict(op=op, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 131072), Hq=hkv * group, Hkv=hkv, d=d,
                 rot=rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)]),
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), interleaved=rng.random() < 0.5,
                 positions=rng.choice(["rows", "given", "far", "striped"]), P=1,
                 scaled=rng.choice([1.0, 1.0, 4.0, 16.0]))
        if c["positions"] == "striped":
            c["P"] = rng.choice([2, 4, 8])
            c["N"] = c["P"] * -(-c["N"] // c["P"])
        most = 131072 * (32 if "rotary" in op else 20 if op == "norm_step" else 32) * 128
        if c["B"] * c["N"] * (c["Hq"] + hkv) * d * (2 if c["dtype"] == "fp32" else 1) <= most:
            return c


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _clip_sizes(tensors, elements):
    """Sizes as a stack of layers has them: every fourth tensor a matrix, the others
    vectors; they sum to `elements`."""
    small = max(1, min(1031, elements // (4 * tensors)))
    sizes = [small + (i % 7) if i % 4 else 0 for i in range(tensors)]
    matrices = sizes.count(0)
    rest = max(matrices, elements - sum(sizes))
    share = rest // matrices
    return [s or share + (i % 5) for i, s in enumerate(sizes)]


def prepare(case, seed):
    g = _generator(seed)
    t = TYPES[case["dtype"]]
    op = case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if op == "clip":
        # gradients in one flat buffer, as a training program accumulates them; the
        # tensors are views of it, of odd sizes, and so are the clipped ones
        sizes = _clip_sizes(case["tensors"], case["elements"])
        total = sum(sizes)
        flat = torch.empty(total, device="cuda", dtype=t)
        grads = list(flat.split(sizes))
        for i, x in enumerate(grads):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float32 if t == torch.float32 else t))
            x.mul_(10.0 ** (-3 + i % 3))
        out = torch.empty_like(flat)
        return {"op": op, "flat": flat, "grads": grads, "out": out, "outs": list(out.split(sizes)), "max_norm": 0.5}
    if op in ("cross", "cross_step"):
        B, Nq, Nkv, Hq, Hkv, d = (case[k] for k in ("B", "Nq", "Nkv", "Hq", "Hkv", "d"))
        k = randn(B, Nkv, Hkv, d)
        q = randn(B, Nq, Hq, d)
        # a trained layer's queries look at some of the keys: each leans towards one
        pick = torch.randint(0, Nkv, (B, Nq, Hkv), generator=g, device="cuda")
        at = k.gather(1, pick[..., None].expand(B, Nq, Hkv, d))
        q += 0.5 * torch.rand((B, Nq, Hq, 1), generator=g, device="cuda") * at.repeat_interleave(Hq // Hkv, dim=2)
        s = {"op": op, "q": q.to(t), "k": k.to(t), "v": randn(B, Nkv, Hkv, d).to(t), "kv_len": None,
             "scale": d ** -0.5}
        if case["ragged"]:
            s["kv_len"] = torch.randint(0, Nkv + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            if B > 1:
                s["kv_len"][B // 2] = 0 if B > 2 else Nkv
                s["kv_len"][0] = Nkv
        if op == "cross_step":
            s["do"] = randn(B, Nq, Hq, d).to(t)
        return s
    B, N, Hq, Hkv, d, rot = (case[k] for k in ("B", "N", "Hq", "Hkv", "d", "rot"))
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if case["scaled"] > 1:  # pairs that turn less than once in the trained length are slowed down
        freq = torch.where(freq * 8192 < 2 * math.pi, freq / case["scaled"], freq)
    s = {"op": op, "q": randn(B, N, Hq, d).to(t), "k": randn(B, N, Hkv, d).to(t), "freq": freq, "P": case["P"],
         "amplitude": 1 + 0.1 * math.log(case["scaled"]), "interleaved": case["interleaved"],
         "striped": case["positions"] == "striped", "positions": None}
    if case["positions"] == "given":  # packed documents: positions start again
        s["positions"] = (torch.arange(N, device="cuda") % max(1, N // 3)).repeat(B, 1)
    elif case["positions"] == "far":  # every sequence has come to a place of its own
        s["positions"] = torch.randint(0, 2 ** 20, (B, 1), generator=g, device="cuda") + torch.arange(N, device="cuda")
    if op in ("norm", "norm_step"):
        # activations before the norm differ in size from channel to channel
        s["q"] = (s["q"].float() * torch.exp(randn(d))).to(t)
        s["k"] = (s["k"].float() * torch.exp(randn(d))).to(t)
        s["qw"], s["kw"] = (1 + 0.2 * randn(d)).to(t), (1 + 0.2 * randn(d)).to(t)
    if op == "norm_step":
        s["dq"], s["dk"] = randn(B, N, Hq, d).to(t), randn(B, N, Hkv, d).to(t)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s, N, dev):
    """Positions [B or 1, N] of the rows, in 64 bits."""
    if s["positions"] is not None:
        return s["positions"]
    row = torch.arange(N, device=dev)
    if s["striped"]:  # host i's row l is position l P + i
        S = N // s["P"]
        row = row % S * s["P"] + row // S
    return row[None]


def _plain_angles(s, N):
    a = _positions(s, N, s["q"].device)[..., None].double() * s["freq"]  # [B or 1, N, rot / 2]
    return (torch.cos(a) * s["amplitude"]).float()[:, :, None], (torch.sin(a) * s["amplitude"]).float()[:, :, None]


def _plain_rotate(x, c, sn, interleaved):
    """x fp32 [B, N, H, d], its first 2 n columns rotated; a new tensor."""
    n = c.shape[-1]
    first, second = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    one, two = first * c - second * sn, first * sn + second * c
    turned = torch.stack((one, two), dim=-1).flatten(-2) if interleaved else torch.cat((one, two), dim=-1)
    return torch.cat((turned, x[..., 2 * n:]), dim=-1)


def _plain_norm_backward(x, w, dy, c, sn, interleaved):
    x, w = x.float(), w.float()
    g = _plain_rotate(dy.float(), c, -sn, interleaved)
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + NORM_EPS)
    x = x * r
    dw = (g * x).sum(dim=(0, 1, 2))
    g = g * w
    return r * (g - x * (g * x).mean(dim=-1, keepdim=True)), dw


def _plain_cross(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    B, Nq, Hq, d = q.shape
    Nkv, Hkv = k.shape[1:3]
    q = q.view(B, Nq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)  # rows (group, query)
    k, v = k.transpose(1, 2), v.transpose(1, 2)
    z = (q @ k.transpose(2, 3)).mul_(s["scale"])
    if s["kv_len"] is not None:
        gone = torch.arange(Nkv, device=z.device) >= s["kv_len"][:, None]
        z.masked_fill_(gone[:, None, None], -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    return q, k, v, p, p @ v, (top + torch.log(total))[..., 0]


def _heads_last(x, B, Nq, Hq, d):
    """[B, Hkv, group * Nq, d] -> [B, Nq, Hq, d]"""
    return x.view(B, Hq, Nq, d).transpose(1, 2).contiguous()


def _plain(s):
    op = s["op"]
    if op == "clip":
        x = s["flat"].float()
        norm = x.square().sum(dtype=torch.float64).sqrt()
        return {"norm": norm.float(),
                "clipped": (x * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0).float()).to(s["flat"].dtype)}
    if op in ("cross", "cross_step"):
        t, (B, Nq, Hq, d) = s["q"].dtype, s["q"].shape
        q, k, v, p, o, lse = _plain_cross(s)
        out = {"o": _heads_last(o, B, Nq, Hq, d).to(t), "lse": lse.reshape(B, Hq, Nq)}
        if op == "cross":
            return out
        do = s["do"].float().transpose(1, 2).reshape(q.shape)
        dv = p.transpose(2, 3) @ do
        dz = (do @ v.transpose(2, 3)).sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p).mul_(s["scale"])
        return dict(out, dq=_heads_last(dz @ k, B, Nq, Hq, d).to(t),
                    dk=(dz.transpose(2, 3) @ q).transpose(1, 2).to(t).contiguous(),
                    dv=dv.transpose(1, 2).to(t).contiguous())
    t, N = s["q"].dtype, s["q"].shape[1]
    c, sn = _plain_angles(s, N)
    if op == "rotary_grad":
        sn = -sn
    if op in ("rotary", "rotary_grad"):
        return {"q": _plain_rotate(s["q"].float(), c, sn, s["interleaved"]).to(t),
                "k": _plain_rotate(s["k"].float(), c, sn, s["interleaved"]).to(t)}

    def forward(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + NORM_EPS) * w.float()
        return _plain_rotate(x, c, sn, s["interleaved"]).to(t)

    out = {"q": forward(s["q"], s["qw"]), "k": forward(s["k"], s["kw"])}
    if op == "norm":
        return out
    dq, dqw = _plain_norm_backward(s["q"], s["qw"], s["dq"], c, sn, s["interleaved"])
    dk, dkw = _plain_norm_backward(s["k"], s["kw"], s["dk"], c, sn, s["interleaved"])
    return dict(out, dq=dq.to(t), dk=dk.to(t), dqw=dqw, dkw=dkw)


def run(state):
    if not own:
        return _plain(state)
    import blockwise_exact_attention_ra_gb300 as ra
    s, op = state, state["op"]
    if op == "clip":
        return {"norm": ra.grad_clip(s["grads"], s["max_norm"], outs=s["outs"], eps=CLIP_EPS), "clipped": s["out"]}
    if op in ("cross", "cross_step"):
        t = s["q"].dtype
        o, lse = ra.cross_attention_fwd(s["q"], s["k"], s["v"], kv_len=s["kv_len"], scale=s["scale"], o_dtype=t)
        if op == "cross":
            return {"o": o, "lse": lse}
        dq, dk, dv = ra.cross_attention_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], kv_len=s["kv_len"],
                                            scale=s["scale"], grad_dtype=t)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    where = dict(positions=s["positions"], interleaved=s["interleaved"], amplitude=s["amplitude"], P=s["P"],
                 striped=s["striped"])
    if op == "rotary":
        q, k = ra.rotary_fwd(s["q"], s["k"], s["freq"], **where)
        return {"q": q, "k": k}
    if op == "rotary_grad":
        q, k = ra.rotary_bwd(s["q"], s["k"], s["freq"], **where)
        return {"q": q, "k": k}
    q, k = ra.norm_rotary_fwd(s["q"], s["k"], s["qw"], s["kw"], s["freq"], eps=NORM_EPS, **where)
    if op == "norm":
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = ra.norm_rotary_bwd(s["q"], s["k"], s["dq"], s["dk"], s["qw"], s["kw"], s["freq"], eps=NORM_EPS,
                                          grad_dtype=s["q"].dtype, **where)
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "clip":
        n = sum(_clip_sizes(case["tensors"], case["elements"]))
        return {"bytes": 2.0 * n * size + 4, "flops": 3.0 * n}
    if op in ("cross", "cross_step"):
        B, Nq, Nkv, Hq, Hkv, d = (case[k] for k in ("B", "Nq", "Nkv", "Hq", "Hkv", "d"))
        # of a ragged batch half of the keys are there on average
        share = 0.5 if case["ragged"] and B > 1 else 1.0
        qs, ks, pairs = B * Nq * Hq * d * size, share * B * Nkv * Hkv * d * size, share * B * Hq * Nq * Nkv * d
        if op == "cross":
            return {"bytes": 2 * qs + 2 * ks + 4.0 * B * Hq * Nq, "flops": 4.0 * pairs}
        # q, do, k, v in; o, dq, dk, dv out; the two products of the forward pass, five of the backward's
        return {"bytes": 4 * qs + 4 * ks + 4.0 * B * Hq * Nq, "flops": 14.0 * pairs}
    B, N, Hq, Hkv, d, rot = (case[k] for k in ("B", "N", "Hq", "Hkv", "d", "rot"))
    n = float(B * N * (Hq + Hkv)) * d
    positions = 8.0 * B * N if case["positions"] in ("given", "far") else 0.0
    if op in ("rotary", "rotary_grad"):
        return {"bytes": 2 * n * size + positions, "flops": 3 * n * rot / d}
    if op == "norm":
        return {"bytes": 2 * n * size + positions, "flops": 4 * n + 3 * n * rot / d}
    # in: q, k and their gradients; out: the normed ones, the gradients of q and k
    return {"bytes": 4 * n * size + positions, "flops": 14 * n + 6 * n * rot / d}


# ------------------------------------------------------------ definition, 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("cross", "cross_step") and work(case)["flops"] > 4e12:  # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for x in s["grads"]:
            total += torch.linalg.vector_norm(x.double()) ** 2
        norm = float(total) ** 0.5
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "clipped": s["flat"].double() * min(1.0, s["max_norm"] / (norm + CLIP_EPS))}
    if op in ("cross", "cross_step"):
        return _exact_cross(s, op == "cross_step")
    B, N, _, d = s["q"].shape
    rot = case["rot"]
    # the pairs as complex numbers, turned by e^{i p f}
    if s["positions"] is not None:
        place = s["positions"].double()
    elif s["striped"]:
        place = torch.arange(N, device="cuda").view(N // s["P"], s["P"]).T.reshape(1, N).double()
    else:
        place = torch.arange(N, device="cuda").view(1, N).double()

    def turned(x, sign):  # one batch entry and head at a time would be slow; one batch entry is not
        y = x.clone()
        for b in range(x.shape[0]):
            e = torch.polar(torch.full((), s["amplitude"], dtype=torch.float64, device="cuda"),
                            sign * place[b % place.shape[0], :, None] * s["freq"])[:, None]
            if case["interleaved"]:
                z = torch.view_as_complex(x[b, ..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * e
                y[b, ..., :rot] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[b, ..., :rot // 2].contiguous(), x[b, ..., rot // 2:rot].contiguous()) * e
                y[b, ..., :rot // 2], y[b, ..., rot // 2:rot] = z.real, z.imag
        return y

    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if op in ("rotary", "rotary_grad"):
            out[name] = turned(x, 1.0 if op == "rotary" else -1.0)
            continue
        w = s[name + "w"].double()
        rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + NORM_EPS) ** 0.5
        out[name] = turned(x / rms * w, 1.0)
        if op == "norm_step":
            dn = turned(s["d" + name].double(), -1.0)
            out[f"d{name}w"] = torch.einsum("bnhc,bnhc->c", dn, x / rms)
            dn *= w
            along = torch.einsum("bnhc,bnhc->bnh", dn, x)[..., None]
            out["d" + name] = dn / rms - x * along / (d * rms ** 3)
    return out


def _exact_cross(s, step):
    B, Nq, Hq, d = s["q"].shape
    Nkv, Hkv = s["k"].shape[1:3]
    names = ("o", "dq", "dk", "dv") if step else ("o",)
    like = {"o": "q", "dq": "q", "dk": "k", "dv": "k"}
    out = {n: torch.zeros(s[like[n]].shape, dtype=torch.float64, device="cuda") for n in names}
    out["lse"] = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = Nkv if s["kv_len"] is None else int(s["kv_len"][b])
        if n == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = s["k"][b, :n, g].double(), s["v"][b, :n, g].double()
            for r in range(0, Nq, 2048):
                rows = slice(r, min(Nq, r + 2048))
                q = s["q"][b, rows, h].double()
                z = q @ k.T * s["scale"]
                out["lse"][b, h, rows] = torch.logsumexp(z, dim=1)
                p = torch.softmax(z, dim=1)
                out["o"][b, rows, h] = p @ v
                if step:
                    do = s["do"][b, rows, h].double()
                    out["dv"][b, :n, g] += p.T @ do
                    dp = do @ v.T
                    ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None]) * s["scale"]
                    out["dq"][b, rows, h] = ds @ k
                    out["dk"][b, :n, g] += ds.T @ q
    return out
