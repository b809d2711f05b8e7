"""Cases for the operators that open and close a training step's backward pass:
the softmax cross entropy of a large vocabulary (the head of the model: hidden
states against the vocabulary's weights, without ever holding the logits) with
its gradients, and the Newton-Schulz orthogonalisation of a weight gradient
that the update of a hidden layer's matrix uses.

A case is one call (`op` "loss": the loss alone, as evaluation and scoring call
it; "step": the loss and its gradients, as a training step calls it; "update":
one orthogonalised update).  With ``own`` false, ``run`` computes the plain form
in 32 bits from elementary torch operations; with ``own`` true it calls the
framework's operators."""
import math

import torch

own = False

IGNORE = -100                        # the target of a token that carries no loss
STEPS, COEFFS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # scoring one token: the weights are read for a single row, latency and bandwidth
        dict(name="loss one token", op="loss", T=1, D=2048, V=32768, dtype="bf16", ignored=0.0),
        # scoring a short ragged prompt with a vocabulary of odd size, fp16
        dict(name="loss ragged fp16", op="loss", T=333, D=1000, V=50021, dtype="fp16", ignored=0.0),
        # perplexity of one block of a long document, large vocabulary
        dict(name="loss long block", op="loss", T=8192, D=2048, V=131072, dtype="bf16", ignored=0.0),
        # the smallest training step: a toy model's head
        dict(name="step small", op="step", T=128, D=256, V=1024, dtype="bf16", ignored=0.0, block=1024),
        # fine-tuning on odd sizes in fp16 with a scaled loss; prompts carry no loss
        dict(name="step ragged fp16", op="step", T=777, D=520, V=10007, dtype="fp16", ignored=0.4, block=4096),
        # an ordinary training step, a third of the tokens are prompt
        dict(name="step ordinary", op="step", T=4096, D=2048, V=32768, dtype="bf16", ignored=0.3, block=8192),
        # a training step with a large vocabulary, in pieces of it
        dict(name="step large vocabulary", op="step", T=4096, D=2048, V=131072, dtype="bf16", ignored=0.0, block=16384),
        # the update of one small projection: latency of the chain of products
        dict(name="update small", op="update", batch=1, rows=128, cols=512, dtype="fp32"),
        # a tall matrix of odd sizes
        dict(name="update ragged", op="update", batch=1, rows=1000, cols=333, dtype="bf16"),
        # a stack of equal small projections (one per head), one call
        dict(name="update stack of heads", op="update", batch=16, rows=256, cols=1024, dtype="fp16"),
        # the square projections of four layers, one call
        dict(name="update stack of layers", op="update", batch=4, rows=2048, cols=2048, dtype="bf16"),
        # the feed-forward layer's W1 with the fp32 gradient its backward pass returns
        dict(name="update feed-forward", op="update", batch=1, rows=8192, cols=2048, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "step", "update"])
    if op == "update":
        # 4 * 2048^3 is the work of the largest listed call's products, per step
        while True:
            b = rng.choice([1, 1, 2, 3, 6])
            m, n = _log_int(rng, 32, 8192), _log_int(rng, 32, 8192)
            k = min(m, n)
            if b * (3 * k * k * max(m, n) + k ** 3) <= 4 * (3 + 1) * 2048 ** 3 and b * m * n <= 2 ** 24:
                return dict(op=op, batch=b, rows=m, cols=n, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    most = 2 ** 13 * 2 ** 11 * 2 ** 17 if op == "loss" else 2 ** 12 * 2 ** 11 * 2 ** 17
    while True:
        T, D, V = _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 512), _log_int(rng, 500, 131072)
        if T * D * V <= most and T * V <= 2 ** 30 and D * V <= 2 ** 28:
            break
    c = dict(op=op, T=T, D=D, V=V, dtype=rng.choice(["bf16", "fp16"]), ignored=rng.choice([0.0, 0.0, 0.25, 0.6]))
    if op == "step":
        c["block"] = rng.choice([V, 2048, 5000, 8192, 16384])
    return c


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    g = _generator(seed)
    t = TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "update":
        # the gradient of a weight: a sum over tokens of outer products, the tokens of
        # unequal weight and the activations with a common direction
        b, m, n, tokens = case["batch"], case["rows"], case["cols"], 4096
        grad = torch.empty(b, m, n, device="cuda", dtype=t)
        for i in range(b):
            dy = randn(tokens, m) * torch.exp(randn(tokens, 1))
            x = randn(tokens, n) + 0.5 * randn(1, n)
            grad[i] = (dy.T @ x / tokens).to(t)
        return {"op": "update", "g": grad[0] if b == 1 else grad}
    T, D, V = case["T"], case["D"], case["V"]
    w = randn(V, D) * (1.5 / math.sqrt(D))
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    # hidden states of a partly trained model: each token leans towards its target's
    # weights, some so far that its probability is near one
    lean = 12.0 * torch.rand((T, 1), generator=g, device="cuda")
    wy = w[y]
    x = randn(T, D) + lean * wy / wy.norm(dim=1, keepdim=True)
    drop = torch.rand((T,), generator=g, device="cuda") < case["ignored"]
    y = torch.where(drop, torch.full_like(y, IGNORE), y)
    state = {"op": case["op"], "x": x.to(t), "w": w.to(t), "y": y}
    if case["op"] == "step":
        # gradient of the mean loss, tokens weighted; fp16 training scales its loss
        scale = 4096.0 if case["dtype"] == "fp16" else 1.0
        weight = 0.5 + torch.rand((T,), generator=g, device="cuda")
        state["dloss"] = weight * (scale / max(1, T))
        state["block"] = min(case["block"], V)
    return state


# ------------------------------------------------------------------ plain forms
def _plain_loss(x, w, y):
    z = x.float() @ w.float().T
    top = z.amax(dim=1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    kept = y != IGNORE
    at = torch.where(kept, y, torch.zeros_like(y))[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    return z, kept, at, loss, lse


def _plain_step(x, w, y, dloss):
    z, kept, at, loss, lse = _plain_loss(x, w, y)
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    d *= torch.where(kept, dloss, torch.zeros_like(dloss))[:, None]
    dx = (d @ w.float()).to(x.dtype)
    dw = (d.T @ x.float()).to(w.dtype)
    return loss, lse, dx, dw


def _plain_update(g):
    a, b, c = COEFFS
    x = g.float()
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1)
    for _ in range(STEPS):
        s = x @ x.transpose(-2, -1)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(-2, -1) if tall else x


def run(state):
    if own:
        import blockwise_exact_attention_ra_gb300 as ra
        if state["op"] == "update":
            return ra.newton_schulz(state["g"], steps=STEPS, coeffs=COEFFS, eps=EPS, out_dtype=torch.bfloat16)
        loss, lse = ra.xent_fwd(state["x"], state["w"], state["y"], ignore_index=IGNORE)
        if state["op"] == "loss":
            return {"loss": loss, "lse": lse}
        dx, dw = ra.xent_bwd(state["x"], state["w"], state["y"], lse, state["dloss"], block=state["block"],
                             dx_dtype=state["x"].dtype, dw_dtype=state["w"].dtype, ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    if state["op"] == "update":
        return _plain_update(state["g"]).to(torch.bfloat16)  # an update is applied in bf16
    if state["op"] == "loss":
        _, _, _, loss, lse = _plain_loss(state["x"], state["w"], state["y"])
        return {"loss": loss, "lse": lse}
    loss, lse, dx, dw = _plain_step(state["x"], state["w"], state["y"], state["dloss"])
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def work(case):
    if case["op"] == "update":
        b, m, n = case["batch"], case["rows"], case["cols"]
        k, l = min(m, n), max(m, n)
        size = 4 if case["dtype"] == "fp32" else 2
        # two symmetric products (half of each) and a full one, each step
        return {"bytes": b * m * n * (size + 2), "flops": STEPS * b * (3.0 * k * k * l + k ** 3)}
    T, D, V = case["T"], case["D"], case["V"]
    bytes_, flops = 2 * (T + V) * D + 8 * T + 8 * T, 2.0 * T * D * V
    if case["op"] == "step":
        # the logits once, and the two products of their gradient
        return {"bytes": bytes_ + 4 * T + 2 * (T + V) * D, "flops": 3 * flops}
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------ definition, 64 bits
def exact(case, seed):
    w = work(case)["flops"] * (2 if case["op"] == "update" else 1)
    if w > 9e12:  # over about 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    if case["op"] == "update":
        a, b, c = COEFFS
        whole = s["g"].double()
        single = whole.dim() == 2
        outs = []
        for x in ([whole] if single else list(whole)):
            x = x / (torch.linalg.norm(x) + EPS)
            for _ in range(STEPS):
                # on whichever side is the smaller: p(X) = a X + b (X X^T) X + c (X X^T)^2 X
                if x.shape[0] <= x.shape[1]:
                    q = x @ x.T
                    qx = q @ x
                    x = a * x + b * qx + c * (q @ qx)
                else:
                    q = x.T @ x
                    xq = x @ q
                    x = a * x + b * xq + c * (xq @ q)
            outs.append(x)
        return outs[0] if single else torch.stack(outs)
    x, w, y = s["x"].double(), s["w"].double(), s["y"]
    T = x.shape[0]
    loss, lse = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for t0 in range(0, T, 1024):
        rows = slice(t0, min(T, t0 + 1024))
        z = x[rows] @ w.T
        lse[rows] = torch.logsumexp(z, dim=1)
        counted = torch.nonzero(y[rows] != IGNORE)[:, 0]
        cls = y[rows][counted]
        loss[t0 + counted] = lse[t0 + counted] - z[counted, cls]
        if case["op"] == "step":
            soft = torch.zeros_like(z)
            soft[counted] = torch.softmax(z[counted], dim=1)
            soft[counted, cls] -= 1.0
            soft *= s["dloss"][rows].double()[:, None]
            dx[rows] = soft @ w
            dw += soft.T @ x[rows]
    out = {"loss": loss, "lse": lse}
    return dict(out, dx=dx, dw=dw) if case["op"] == "step" else out
