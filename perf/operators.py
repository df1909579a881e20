"""Cases for the layer operators: the 8-bit product with token and channel scales, the norms around a block with its
gate and residual scale, and the cross entropy over a large vocabulary with its gradient.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once), or, where `own` is true,
through the package's calls.  `exact` computes the same from the definitions in fp64.
"""

import math

import torch

own = False

BF16, F16, F32 = "bfloat16", "float16", "float32"
SIZE = {BF16: 2, F16: 2, F32: 4}
LARGEST = 6.7e12  # flops of the largest listed case


def listed():
    return [
        # One decoded token through a 4096 x 4096 layer: latency, and one read of the codes.
        {"name": "matmul one token", "op": "matmul", "T": 1, "K": 4096, "N": 4096, "dtype": BF16, "bias": False},
        # A decode batch through the down projection of a 14336-wide block.
        {"name": "matmul 40 sequences", "op": "matmul", "T": 40, "K": 14336, "N": 4096, "dtype": BF16, "bias": True},
        # Odd sizes in every direction, fp32 in and out.
        {"name": "matmul odd sizes", "op": "matmul", "T": 333, "K": 4099, "N": 1999, "dtype": F32, "bias": True},
        # A prompt of 4096 tokens through the up projection of a 14336-wide block.
        {"name": "matmul 4096 tokens", "op": "matmul", "T": 4096, "K": 4096, "N": 14336, "dtype": F16, "bias": False},
        # The end of a block for one decoded token: its norm, gate and residual, then the next block's norm.
        {"name": "norm one token", "op": "norm", "T": 1, "D": 4096, "dtype": BF16, "kind": "rms", "groups": 0},
        # The same for 8 sequences of 1024 tokens with a gate row for each sequence.
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "D": 4096, "dtype": BF16, "kind": "rms", "groups": 8},
        # Backward pass of that over 16384 tokens, gate rows for 8 sequences.
        {"name": "norm backward 16384", "op": "norm_backward", "T": 16384, "D": 4096, "dtype": BF16, "kind": "rms", "groups": 8},
        # Backward pass of layer norms of an odd width in fp32, one gate row for all tokens.
        {"name": "norm backward odd", "op": "norm_backward", "T": 1531, "D": 1999, "dtype": F32, "kind": "layer", "groups": 1},
        # The norm's output as 8-bit codes, straight into the next layer's product.
        {"name": "norm to matmul", "op": "norm_matmul", "T": 512, "D": 4096, "N": 4096, "dtype": BF16, "kind": "rms", "groups": 1},
        # The loss of a short evaluation text under a small head.
        {"name": "loss 200 tokens", "op": "loss", "T": 200, "D": 1024, "V": 32768, "dtype": BF16},
        # Loss and gradient with an odd vocabulary in fp16.
        {"name": "loss gradient odd", "op": "loss_gradient", "T": 1021, "D": 1000, "V": 50021, "dtype": F16},
        # Loss and gradient of a calibration batch of 2048 tokens over a vocabulary of 131072.
        {"name": "loss gradient 2048", "op": "loss_gradient", "T": 2048, "D": 4096, "V": 131072, "dtype": BF16},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "norm", "norm_backward", "norm_matmul", "loss", "loss_gradient"])
    while True:
        c = {"op": op, "T": _spread(rng, 1, 4096), "dtype": rng.choice([BF16, BF16, F16, F32])}
        if op == "matmul":
            c |= {"K": _spread(rng, 64, 14336), "N": _spread(rng, 64, 14336), "bias": rng.random() < 0.5}
        elif op.startswith("norm"):
            groups = rng.choice([0, 1, 1, 2, 5])
            each = _spread(rng, 1, 16384) // max(1, groups)
            c |= {"T": max(1, each) * max(1, groups), "D": _spread(rng, 64, 14336), "kind": rng.choice(["rms", "layer"]), "groups": groups}
            if op == "norm_matmul":
                c |= {"T": max(1, each // 4) * max(1, groups), "N": _spread(rng, 64, 14336)}
        else:
            c |= {"D": _spread(rng, 128, 4096), "V": _spread(rng, 1000, 131072)}
            c["dtype"] = rng.choice([BF16, F16])
        if rng.random() < 0.5:  # sizes that a matrix of a model has, in multiples of 64; else whatever came
            c |= {k: max(64, c[k] // 64 * 64) for k in ("K", "N", "D", "V") if k in c}
        if work(c)["flops"] <= LARGEST and not any(c.get(k) == 3 * 1024 for k in "TKNDV") and work(c)["bytes"] < 2e9:
            return c


def work(c):
    T, e = c["T"], SIZE[c["dtype"]]
    if c["op"] == "matmul":
        K, N = c["K"], c["N"]
        return {"bytes": T * K * e + N * K + 4 * N * (1 + c["bias"]) + T * N * e, "flops": 2 * T * K * N}
    D = c["D"]
    gate = max(0, c.get("groups", 0)) * D
    if c["op"] == "norm":  # x, h read, y, z written; two weights (with biases), the gate
        return {"bytes": 4 * T * D * e + 4 * _weights(c) * D + gate * e, "flops": 12 * T * D}
    if c["op"] == "norm_backward":  # dy, dz, y, h read, dx, dh written; weights and gate, and their gradients
        return {"bytes": 6 * T * D * e + 8 * _weights(c) * D + gate * (e + 4), "flops": 30 * T * D}
    if c["op"] == "norm_matmul":  # x, h read, y and the product written, codes kept on the chip
        N = c["N"]
        return {"bytes": 3 * T * D * e + 4 * _weights(c) * D + gate * e + N * D + 4 * N + T * N * e, "flops": 2 * T * D * N}
    V = c["V"]
    if c["op"] == "loss":
        return {"bytes": (T + V) * D * e + 16 * T, "flops": 2 * T * V * D}
    return {"bytes": 2 * (T + V) * D * e + 20 * T, "flops": 6 * T * V * D}


def _weights(c):
    return 2 if c["kind"] == "rms" else 4


def _codes_and_scales(N, K, gen):
    """8-bit codes of a weight matrix, about Gaussian with clipped tails, and one scale for each output."""
    w = torch.empty((N, K), dtype=torch.int8, device="cuda")
    for lo in range(0, N, 4096):  # in pieces: the draws are in fp32
        w[lo : lo + 4096] = (torch.randn((min(4096, N - lo), K), generator=gen, device="cuda") * 34).round_().clamp_(-127, 127)
    return w, (0.5 + torch.rand(N, generator=gen, device="cuda")) * (0.02 / 34)


def _activations(T, D, dtype, gen):
    """Activations with a few loud features, as a residual stream has them."""
    loud = 1 + 7 * (torch.rand(D, generator=gen, device="cuda") < 0.01)
    return (torch.randn((T, D), generator=gen, device="cuda") * loud).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    s, T = {"case": case}, case["T"]
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "matmul":
        s["x"] = _activations(T, case["K"], dtype, gen)
        s["w"], s["ws"] = _codes_and_scales(case["N"], case["K"], gen)
        s["bias"] = 0.1 * rand(case["N"]) if case["bias"] else None
    elif case["op"].startswith("norm"):
        D, groups = case["D"], case["groups"]
        s["h"] = _activations(T, D, dtype, gen)
        s["post"], s["pre"] = 1 + 0.1 * rand(D), 1 + 0.1 * rand(D)
        layer = case["kind"] == "layer"
        s["post_bias"], s["pre_bias"] = (0.1 * rand(D) if layer else None), (0.1 * rand(D) if layer else None)
        s["gate"] = None if not groups else (0.3 * rand(groups, D)).to(dtype)
        s["alpha"], s["eps"] = 0.9, 1e-5
        if case["op"] == "norm_backward":
            s["y"] = _activations(T, D, dtype, gen)
            s["dy"], s["dz"] = (0.01 * rand(T, D)).to(dtype), (0.01 * rand(T, D)).to(dtype)
        else:
            s["x"] = _activations(T, D, dtype, gen)
        if case["op"] == "norm_matmul":
            s["w"], s["ws"] = _codes_and_scales(case["N"], D, gen)
    else:
        D, V = case["D"], case["V"]
        s["w"] = torch.empty((V, D), dtype=dtype, device="cuda")
        for lo in range(0, V, 16384):
            s["w"][lo : lo + 16384] = (rand(min(16384, V - lo), D) * D ** -0.5).to(dtype)
        # Hidden states that lean towards their target, so that losses are those of a model that has learnt something;
        # one token in 16 or so has no target.
        y = torch.randint(0, V, (T,), generator=gen, device="cuda")
        s["h"] = (rand(T, D) + (2 + 4 * torch.rand((T, 1), generator=gen, device="cuda")) * s["w"][y].float()).to(dtype)
        s["target"] = torch.where(torch.rand(T, generator=gen, device="cuda") < 1 / 16, -100, y)
    return s


# ------------------------------------------------------------------ the plain forms


def _quantize(x):
    """Codes and scales of each token: s = max |x| / 127, code = x / s rounded to nearest, ties to even."""
    top = x.abs().amax(1)
    scale = top / torch.full_like(top, 127.0)
    return torch.round(x / torch.where(scale > 0, scale, 1)[:, None]).clamp(-127, 127), scale


def _matmul(codes, scale, w, ws, bias):
    y = (codes @ w.float().t()) * scale[:, None] * ws
    return y if bias is None else y + bias


def _norm(x, w, b, eps, kind):
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    n = c * torch.rsqrt(c.square().mean(1, keepdim=True) + eps) * w
    return n if b is None else n + b


def _per_token(gate, T):
    return 1.0 if gate is None else gate.float().repeat_interleave(T // gate.shape[0], 0)


def _norm_residual(s, kind):
    x, h = s["x"].float(), s["h"].float()
    u = _norm(h, s["post"], s["post_bias"], s["eps"], kind)
    y = s["alpha"] * x + _per_token(s["gate"], len(x)) * u
    return y, _norm(y, s["pre"], s["pre_bias"], s["eps"], kind)


def _norm_gradients(x, w, dn, eps, kind):
    """Gradients of a norm's input, weight and bias for its output's gradient dn."""
    c = x - x.mean(1, keepdim=True) if kind == "layer" else x
    r = torch.rsqrt(c.square().mean(1, keepdim=True) + eps)
    unit = c * r
    g = dn * w
    dx = g - unit * (g * unit).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return dx * r, (dn * unit).sum(0), dn.sum(0)


def _norm_backward(s, kind):
    dy, dz, y, h = (s[k].float() for k in ("dy", "dz", "y", "h"))
    T, gate = len(y), s["gate"]
    through, dpre, dpre_bias = _norm_gradients(y, s["pre"], dz, s["eps"], kind)
    dy = dy + through
    du = dy * _per_token(gate, T)
    dh, dpost, dpost_bias = _norm_gradients(h, s["post"], du, s["eps"], kind)
    out = {"X": (s["alpha"] * dy).to(s["y"].dtype), "H": dh.to(s["y"].dtype), "post": dpost, "pre": dpre}
    if kind == "layer":
        out |= {"post_bias": dpost_bias, "pre_bias": dpre_bias}
    if gate is not None:
        u = _norm(h, s["post"], s["post_bias"], s["eps"], kind)
        out["gate"] = (dy * u).view(gate.shape[0], -1, h.shape[1]).sum(1)
    return out


def _loss(h, w, target):
    """Losses, log-sums and probabilities: -log softmax(h w^T)[target], 0 where there is no target."""
    logits = h @ w.t()
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = (torch.log(total) + top)[:, 0]
    has = target >= 0
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    return torch.where(has, lse - at, 0.0), lse, e.div_(total), has


def _loss_gradient(h, w, target):
    """Losses, and the gradients of their mean over the tokens with a target."""
    loss, lse, p, has = _loss(h, w, target)
    coef = has.float() / has.sum().clamp(min=1)
    g = p.mul_(coef[:, None])
    g[torch.arange(len(h), device=h.device), target.clamp(min=0)] -= coef
    return loss, lse, g @ w, g.t() @ h


def _plain(s):
    c = s["case"]
    dtype = getattr(torch, c["dtype"])
    if c["op"] == "matmul":
        return _matmul(*_quantize(s["x"].float()), s["w"], s["ws"], s["bias"]).to(dtype)
    if c["op"] == "norm":
        y, z = _norm_residual(s, c["kind"])
        return y.to(dtype), z.to(dtype)
    if c["op"] == "norm_matmul":
        y, z = _norm_residual(s, c["kind"])
        return y.to(dtype), _matmul(*_quantize(z), s["w"], s["ws"], None).to(dtype)
    if c["op"] == "norm_backward":
        return _norm_backward(s, c["kind"])
    if c["op"] == "loss":
        return _loss(s["h"].float(), s["w"].float(), s["target"])[:2]
    loss, lse, dh, dw = _loss_gradient(s["h"].float(), s["w"].float(), s["target"])
    return loss, lse, dh.to(dtype), dw.to(dtype)


# ------------------------------------------------------------------ the package's calls


def _own(s):
    import kronecker_hessian_gptq_gb300 as bk

    c = s["case"]
    if c["op"] == "matmul":
        return bk.int8_matmul(s["x"], s["w"], s["ws"], bias=s["bias"])[0]
    if c["op"].startswith("loss"):
        call = bk.linear_cross_entropy if c["op"] == "loss" else bk.linear_cross_entropy_grad
        return call(s["h"], s["w"], s["target"])[:-1]
    args = {k: s[k] for k in ("post", "gate", "pre", "post_bias", "pre_bias", "alpha", "eps")} | {"kind": c["kind"]}
    if c["op"] == "norm":
        return bk.norm_residual(s["x"], s["h"], **args)
    if c["op"] == "norm_backward":
        return {k: v for k, v in bk.norm_residual_backward(s["dy"], s["dz"], s["y"], s["h"], **args).items() if v is not None}
    y, codes, scale = bk.norm_residual(s["x"], s["h"], **args, codes=True)
    return y, bk.int8_matmul(codes, s["w"], s["ws"], x_scales=scale, dtype=y.dtype)[0]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in fp64


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op, T = case["op"], case["T"]

    def product(x):
        # The scale is an fp32 number by definition; each output is the exact integer sum, scaled.
        scale = (x.abs().max(1).values / 127).float().double()
        codes = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0).round()
        y = torch.empty((T, case["N"]), dtype=torch.float64, device="cuda")
        for lo in range(0, case["N"], 2048):
            part = slice(lo, lo + 2048)
            y[:, part] = (codes @ s["w"][part].double().t()) * d["ws"][part] * scale[:, None]
        return y

    if op == "matmul":
        y = product(d["x"])
        return y + d["bias"] if case["bias"] else y

    def normed(x, w, b):
        if case["kind"] == "layer":
            v, m = torch.var_mean(x, 1, correction=0, keepdim=True)
            return (x - m) / (v + s["eps"]).sqrt() * w + b
        return x / (x.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt() * w

    def gated(h, gate):
        u = normed(h, d["post"], d["post_bias"])
        return u if gate is None else (u.view(gate.shape[0], -1, case["D"]) * gate[:, None]).view(T, -1)

    if op in ("norm", "norm_matmul"):
        y = d["x"] * s["alpha"] + gated(d["h"], d["gate"])
        z = normed(y, d["pre"], d["pre_bias"])
        return y, z if op == "norm" else product(z)

    if op == "norm_backward":
        names = ["post", "gate", "pre", "post_bias", "pre_bias"]
        for k in ["y", "h"] + names:
            if d[k] is not None:
                d[k].requires_grad_()
        out = {}
        z = normed(d["y"], d["pre"], d["pre_bias"])
        to = [k for k in ("y", "pre", "pre_bias") if d[k] is not None]
        out |= dict(zip(to, torch.autograd.grad(z, [d[k] for k in to], d["dz"])))
        total = out.pop("y") + d["dy"]
        to = [k for k in ("h", "post", "post_bias", "gate") if d[k] is not None]
        out |= dict(zip(to, torch.autograd.grad(gated(d["h"], d["gate"]), [d[k] for k in to], total)))
        return {"X": total * s["alpha"], "H": out.pop("h")} | out

    if work(case)["flops"] > 1.5 * LARGEST:
        return None
    h, y, V = d["h"], s["target"], case["V"]
    has = y >= 0
    # The vocabulary in pieces, so that the fp64 logits are never there at once.
    pieces = [slice(lo, min(V, lo + 16384)) for lo in range(0, V, 16384)]
    logits = [h @ s["w"][q].double().t() for q in pieces]
    lse = torch.logsumexp(torch.stack([torch.logsumexp(x, 1) for x in logits]), 0)
    right = (h * s["w"][y.clamp(min=0)].double()).sum(1)
    loss = torch.where(has, lse - right, 0.0)
    if op == "loss":
        return loss, lse
    coef = has.double() / max(1, int(has.sum()))
    dh, dw = torch.zeros_like(h), torch.empty((V, case["D"]), dtype=torch.float64, device="cuda")
    for k, q in enumerate(pieces):
        g = (logits[k] - lse[:, None]).exp_()
        logits[k] = None
        inside = has & (y >= q.start) & (y < q.stop)
        g[inside, y[inside] - q.start] -= 1
        g *= coef[:, None]
        dh += g @ s["w"][q].double()
        dw[q] = g.t() @ h
    return loss, lse, dh, dw
