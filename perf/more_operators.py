"""Cases for the operators of a projection that is trained and run in 8-bit floating point: the product with a scale for
each block of 128 and its gradients, the norms of queries and keys for each head with the position rotation and their
gradients, and the AdamW step over many tensors with states in 32 bits or in 8.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once), or, where `own` is true,
through the package's calls.  `exact` computes the same from the definitions in fp64.
"""

import math

import torch

own = False

BF16, F16, F32 = "bfloat16", "float16", "float32"
SIZE = {BF16: 2, F16: 2, F32: 4}
E4M3, TOP = torch.float8_e4m3fn, 448.0
GROUP = 256  # values that share a scale in 8-bit optimizer states
LARGEST = 4.9e11  # flops of the largest listed product
MOST_BYTES = 4e9  # of the largest listed case


def listed():
    return [
        # One decoded token through a 4096 x 4096 layer: latency, and one read of the codes.
        {"name": "product one token", "op": "product", "T": 1, "K": 4096, "N": 4096, "dtype": BF16, "bias": False},
        # A decode batch through the down projection of a 14336-wide block.
        {"name": "product 40 sequences", "op": "product", "T": 40, "K": 14336, "N": 4096, "dtype": BF16, "bias": True},
        # Odd sizes in every direction, fp32 in and out.
        {"name": "product odd sizes", "op": "product", "T": 333, "K": 4099, "N": 1999, "dtype": F32, "bias": True},
        # A prompt of 4096 tokens through the up projection of a 14336-wide block.
        {"name": "product 4096 tokens", "op": "product", "T": 4096, "K": 4096, "N": 14336, "dtype": BF16, "bias": False},
        # Backward pass of a 4096 x 4096 layer over a training batch of 4096 tokens.
        {"name": "product gradients 4096", "op": "product_gradients", "T": 4096, "K": 4096, "N": 4096, "dtype": BF16},
        # The same at odd sizes in fp16, as a short calibration text gives them.
        {"name": "product gradients odd", "op": "product_gradients", "T": 777, "K": 1000, "N": 2055, "dtype": F16},
        # Queries and keys of one decoded token, 32 and 8 heads of 128.
        {"name": "heads one token", "op": "heads", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "dtype": BF16, "pairs": "halves"},
        # The same for a prompt of 8192 tokens, taken out of the projection's common output.
        {"name": "heads 8192 tokens", "op": "heads", "T": 8192, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "dtype": BF16, "pairs": "halves"},
        # Backward pass of that over 16384 tokens.
        {"name": "heads gradients 16384", "op": "heads_gradients", "T": 16384, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "dtype": BF16,
         "pairs": "halves"},
        # Backward pass with heads of 80 of which 20 are rotated, neighbours in pairs, an odd number of tokens, fp32.
        {"name": "heads gradients part", "op": "heads_gradients", "T": 1531, "Hq": 7, "Hk": 3, "D": 80, "R": 20, "dtype": F32,
         "pairs": "neighbours"},
        # The small parameters of a model (norms, gates, scales): many tensors, little work in each.
        {"name": "adamw small tensors", "op": "adamw", "tensors": 130, "smallest": 64, "largest": 16384, "bits": 32, "dtype": F32,
         "grad": F32, "copy": False},
        # Four matrices of a 14336-wide block: fp32 masters, 8-bit states, bf16 gradients and bf16 copies for the forward pass.
        {"name": "adamw 8 bits large", "op": "adamw", "tensors": 4, "smallest": 4096 * 14336, "largest": 4096 * 14336, "bits": 8,
         "dtype": F32, "grad": BF16, "copy": True},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product_gradients", "heads", "heads_gradients", "adamw"])
    while True:
        c = {"op": op}
        if op.startswith("product"):
            c |= {"T": _spread(rng, 1, 4096), "K": _spread(rng, 64, 14336), "N": _spread(rng, 64, 14336),
                  "dtype": rng.choice([BF16, BF16, F16, F32])}
            if rng.random() < 0.5:  # sizes that a matrix of a model has, in multiples of 64; else whatever came
                c |= {k: c[k] // 64 * 64 for k in "KN"}
            if op == "product":
                c["bias"] = rng.random() < 0.5
        elif op.startswith("heads"):
            hk = rng.choice([1, 2, 3, 4, 8])
            d = rng.choice([64, 80, 96, 128, 192, 256, _spread(rng, 8, 256)])
            r = d if rng.random() < 0.6 else max(2, int(d * rng.choice([0.25, 0.5, 0.75])))
            c |= {"T": _spread(rng, 1, 16384), "Hq": hk * rng.choice([1, 2, 4, 7, 8]), "Hk": hk, "D": d, "R": r // 2 * 2,
                  "dtype": rng.choice([BF16, BF16, F16, F32]), "pairs": rng.choice(["halves", "halves", "neighbours"])}
        else:
            n, a = _spread(rng, 1, 200), _spread(rng, 1, 4096)
            c |= {"tensors": n, "smallest": a, "largest": max(a, _spread(rng, 1000, 4e7)), "bits": rng.choice([8, 32]),
                  "dtype": rng.choice([F32, F32, BF16]), "grad": rng.choice([F32, BF16, F16]), "copy": False}
            c["copy"] = c["dtype"] == F32 and rng.random() < 0.4
        w = work(c)
        if w["flops"] <= LARGEST and w["bytes"] < MOST_BYTES / 2:
            return c


def _sizes(c):
    """Lengths of the tensors of an AdamW case, evenly spread in their logarithm."""
    n, a, b = c["tensors"], c["smallest"], c["largest"]
    return [max(1, int(round(a * (b / a) ** (i / max(1, n - 1))))) for i in range(n)]


def _up(a, b):
    return -(-a // b)


def work(c):
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        each = 2 * SIZE[c["dtype"]] + SIZE[c["grad"]] + 2 * c["copy"] + (4 + 16 / GROUP if c["bits"] == 8 else 16)
        return {"bytes": int(n * each), "flops": 14 * n}
    T, e = c["T"], SIZE[c["dtype"]]
    if c["op"].startswith("product"):
        K, N = c["K"], c["N"]
        weights = N * K + 4 * _up(N, 128) * _up(K, 128)
        if c["op"] == "product":
            return {"bytes": T * K * e + weights + 4 * N * c["bias"] + T * N * e, "flops": 2 * T * K * N}
        # dY, X and the weights read, dX and dW written
        return {"bytes": (T * N + 2 * T * K + N * K) * e + weights, "flops": 4 * T * K * N}
    values = T * (c["Hq"] + c["Hk"]) * c["D"]
    if c["op"] == "heads":
        return {"bytes": 2 * values * e + 8 * T + 4 * c["R"] + 8 * c["D"], "flops": 8 * values}
    return {"bytes": 3 * values * e + 8 * T + 4 * c["R"] + 16 * c["D"], "flops": 18 * values}


def _activations(T, D, dtype, gen):
    """Activations with a few loud features, as a residual stream has them."""
    loud = 1 + 7 * (torch.rand(D, generator=gen, device="cuda") < 0.01)
    return (torch.randn((T, D), generator=gen, device="cuda") * loud).to(dtype)


def _in_rows_of_16(codes):
    """The same codes in rows that start on 16 bytes."""
    n, k = codes.shape
    room = torch.zeros((n, _up(k, 16) * 16), dtype=torch.uint8, device="cuda")
    room[:, :k] = codes.view(torch.uint8)
    return room.view(E4M3)[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    s = {"case": case}
    rand = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"].startswith("product"):
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = _activations(T, K, dtype, gen)
        codes, s["ws"] = _in_blocks(rand(N, K) * (K ** -0.5 * (0.5 + torch.rand((N, 1), generator=gen, device="cuda"))), 128, 128)
        s["w"] = _in_rows_of_16(codes)
        if case["op"] == "product":
            s["bias"] = 0.1 * rand(N) if case["bias"] else None
        else:
            s["dy"] = (0.01 * rand(T, N) * torch.exp(rand(T, 1))).to(dtype)
        return s
    if case["op"].startswith("heads"):
        T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
        qkv = _activations(T, (Hq + 2 * Hk) * D, dtype, gen).view(T, Hq + 2 * Hk, D)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq : Hq + Hk]
        s["qw"], s["kw"] = 1 + 0.2 * rand(D), 1 + 0.2 * rand(D)
        # Sequences of a long context: positions run on from where a chunk of the prompt begins.
        first = torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda")
        s["positions"] = first + torch.arange(T, device="cuda")
        s["freqs"] = 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        s["eps"] = 1e-6
        if case["op"] == "heads_gradients":
            s["dq"], s["dk"] = (0.01 * rand(T, Hq, D)).to(dtype), (0.01 * rand(T, Hk, D)).to(dtype)
        return s
    # AdamW: tensors that lie one after another in flat buffers, each on 256 values.
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, GROUP) * GROUP)
    total = starts[-1]
    cut = lambda flat, per=1: [flat[a // per : a // per + _up(n, per)] for a, n in zip(starts, sizes)]  # noqa: E731
    s["live"] = torch.zeros(total, dtype=torch.bool, device="cuda")
    for part in cut(s["live"]):
        part.fill_(True)
    spread = torch.exp(rand(_up(total, 64))).repeat_interleave(64)[:total]  # gradients differ in size across a matrix
    p = torch.where(s["live"], 0.02 * rand(total), 0.0).to(dtype)
    g = torch.where(s["live"], 1e-3 * spread * rand(total), 0.0).to(getattr(torch, case["grad"]))
    m, v = 3e-4 * spread * rand(total), 1e-6 * spread.square() * (0.5 + torch.rand(total, generator=gen, device="cuda"))
    m, v = torch.where(s["live"], m, 0.0), torch.where(s["live"], v, 0.0)
    del spread
    flat = {"p": p, "g": g}
    if case["bits"] == 32:
        flat |= {"m": m, "v": v}
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            scale = x.view(-1, GROUP).abs().amax(1) / TOP
            inv = torch.where(scale > 0, 1 / scale, 0.0)
            flat[name], flat[name + "_scales"] = (x.view(-1, GROUP) * inv[:, None]).clamp(-TOP, TOP).to(E4M3).view(-1), scale
    s["flat"] = flat
    s["params"], s["grads"] = cut(p), cut(g)
    s["states"] = {k: cut(flat[k], GROUP if k.endswith("scales") else 1) for k in flat if k not in "pg"}
    if case["copy"]:
        flat["copy"] = p.to(torch.bfloat16)
        s["copies"] = cut(flat["copy"])
    s["args"] = {"step": 100 + seed % 1000, "lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1, "grad_scale": 0.5}
    s["seed"] = seed % 1000003
    s["place"] = (starts, sizes)
    return s


# ------------------------------------------------------------------ the plain forms


def _in_blocks(x, rows, cols):
    """Codes of an fp32 matrix in e4m3 with a scale for each block: scale = max |x| / 448, code = x (1 / scale) rounded."""
    T, K = x.shape
    r, c = _up(T, rows), _up(K, cols)
    x = torch.nn.functional.pad(x, (0, c * cols - K, 0, r * rows - T)).view(r, rows, c, cols)
    top = x.abs().amax((1, 3))
    scale = top / torch.full_like(top, TOP)
    inv = torch.where(scale >= 2.0 ** -126, 1 / scale, 0.0)
    codes = (x * inv[:, None, :, None]).clamp(-TOP, TOP).to(E4M3).view(r * rows, c * cols)
    return codes[:T, :K], torch.where(inv > 0, scale, 0.0)


def _values(codes, scale, rows, cols):
    """What codes in blocks stand for, in fp32."""
    T, K = codes.shape
    return codes.float() * scale.repeat_interleave(rows, 0)[:T].repeat_interleave(cols, 1)[:, :K]


def _product(s):
    y = _values(*_in_blocks(s["x"].float(), 1, 128), 1, 128) @ _values(s["w"], s["ws"], 128, 128).t()
    return y if s["bias"] is None else y + s["bias"]


def _product_gradients(s):
    dy, x = s["dy"].float(), s["x"].float()
    dx = _values(*_in_blocks(dy, 1, 128), 1, 128) @ _values(s["w"], s["ws"], 128, 128)
    # The sum over tokens: a scale for each 128 tokens of a column.
    dw = _values(*_in_blocks(dy, 128, 1), 128, 1).t() @ _values(*_in_blocks(x, 128, 1), 128, 1)
    return {"X": dx.to(s["dy"].dtype), "W": dw.to(s["dy"].dtype)}


def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["freqs"]  # in 64 bits: far positions turn many times
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(x, cos, sin, pairs):
    """The first 2 n of the last axis turned by n angles, in pairs (i, i + n) or (2 i, 2 i + 1)."""
    n = cos.shape[-1]
    out = x.clone()
    a, b = (slice(0, n), slice(n, 2 * n)) if pairs == "halves" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _heads(s):
    cos, sin = _cos_sin(s)
    out = []
    for x, w in ((s["q"].float(), s["qw"]), (s["k"].float(), s["kw"])):
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
        out.append(_rotate(n, cos, sin, s["case"]["pairs"]).to(s["q"].dtype))
    return out


def _heads_gradients(s):
    cos, sin = _cos_sin(s)
    out = {}
    for name, dy, x, w in (("Q", s["dq"], s["q"], s["qw"]), ("K", s["dk"], s["k"], s["kw"])):
        dn, x = _rotate(dy.float(), cos, -sin, s["case"]["pairs"]), x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
        unit, g = x * r, dn * w
        out[name] = ((g - unit * (g * unit).mean(-1, keepdim=True)) * r).to(dy.dtype)
        out[name.lower() + "_weight"] = (dn * unit).sum((0, 1))
    return out


def _bits(index, seed, step, tensor):
    """32 random bits for each value: its place in its tensor, mixed with the seed, the step and the tensor's place."""
    low = 0xFFFFFFFF
    key = (seed * 0x9E3779B1 + step * 0x6A09E667 + tensor * 0xBB67AE85) & low
    x = (index * 0x9E3779B1 + (index >> 32) * 0xBB67AE85 + key) & low
    x = ((x ^ (x >> 16)) * 0x6A09E667) & low
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & low
    return x ^ (x >> 16)


def _round_at_random(q, bits):
    """e4m3 of 0 <= q, up with the probability of what is cut off; bits: 16 random ones."""
    u = q.view(torch.int32)
    normal = ((u + (bits.int() << 4)) >> 20) - (120 << 3)
    small = (q * 512 + bits.float() * 2.0 ** -16).int()
    return torch.where(q >= 2.0 ** -6, normal, small).clamp(max=126)


def _adamw(s):
    f, a = s["flat"], s["args"]
    starts, sizes = s["place"]
    t, lr, (b1, b2) = a["step"], a["lr"], a["betas"]
    for i, (start, n) in enumerate(zip(starts, sizes)):
        at = slice(start, start + _up(n, GROUP) * GROUP)  # to the end of the last group: zeros
        groups = slice(start // GROUP, at.stop // GROUP)
        g = f["g"][at].float() * a["grad_scale"]
        m, v = f["m"][at].float(), f["v"][at].float()
        if s["case"]["bits"] == 8:
            m = (m.view(-1, GROUP) * f["m_scales"][groups, None]).view(-1)
            v = (v.view(-1, GROUP) * f["v_scales"][groups, None]).view(-1).square()
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        root = v.sqrt()
        p = f["p"][at].float() * (1 - lr * a["weight_decay"])
        p -= m / (root * (1 / math.sqrt(1 - b2 ** t)) + a["eps"]) * (lr / (1 - b1 ** t))
        f["p"][at] = p.to(f["p"].dtype)
        if "copy" in f:
            f["copy"][at] = p.bfloat16()
        if s["case"]["bits"] == 32:
            f["m"][at], f["v"][at] = m, v
            continue
        bits = _bits(torch.arange(len(p), device=p.device), s["seed"], t, i)
        for name, x, b in (("m", m, bits >> 16), ("v", root, bits & 0xFFFF)):
            top = x.view(-1, GROUP).abs().amax(1)
            scale = top / torch.full_like(top, TOP)
            inv = torch.where(scale >= 2.0 ** -126, 1 / scale, 0.0)
            q = (x.abs().view(-1, GROUP) * inv[:, None]).view(-1)
            code = _round_at_random(q, b)
            # a root that is there stays there: nothing is divided by a lost one
            code = torch.where((q > 0) & (code == 0), 1, code) if name == "v" else code | ((x < 0).int() << 7)
            f[name][at] = code.to(torch.uint8).view(E4M3)
            f[name + "_scales"][groups] = torch.where(inv > 0, scale, 0.0)
    return _of_adamw(f)


def _of_adamw(f):
    return {k: f[k] for k in f if k != "g"}


def _plain(s):
    op = s["case"]["op"]
    if op == "product":
        return _product(s).to(s["x"].dtype)
    return {"product_gradients": _product_gradients, "heads": _heads, "heads_gradients": _heads_gradients, "adamw": _adamw}[op](s)


# ------------------------------------------------------------------ the package's calls


def _own(s):
    import kronecker_hessian_gptq_gb300 as bk

    op = s["case"]["op"]
    if op == "product":
        return bk.fp8_matmul(s["x"], s["w"], s["ws"], bias=s["bias"])[0]
    if op == "product_gradients":
        grads = bk.fp8_matmul_backward(s["dy"], s["x"], s["w"], s["ws"])[0]
        return {"X": grads["X"], "W": grads["W"]}
    if op == "adamw":
        bk.adamw(s["params"], s["grads"], s["states"], copies=s.get("copies"), seed=s["seed"], **s["args"])
        return _of_adamw(s["flat"])
    args = {"q_weight": s["qw"], "k_weight": s["kw"], "eps": s["eps"], "pairs": s["case"]["pairs"]}
    if op == "heads":
        return bk.head_norm_rotary(s["q"], s["k"], s["positions"], s["freqs"], **args)
    return bk.head_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["freqs"], **args)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definitions in fp64


def _e4m3(q):
    """Nearest number of e4m3 to the fp64 q, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-TOP, TOP)


def _block_values(x, rows, cols):
    """The values that the e4m3 codes of x in blocks stand for, the scale and its reciprocal being fp32 numbers."""
    T, K = x.shape
    out = torch.empty_like(x)
    tall = max(rows, 1024)
    for lo in range(0, T, tall):  # in pieces: the steps are in fp64
        part = x[lo : lo + tall]
        t = len(part)
        full = torch.zeros((_up(t, rows) * rows, _up(K, cols) * cols), dtype=torch.float64, device=x.device)
        full[:t, :K] = part
        b = full.view(_up(t, rows), rows, _up(K, cols), cols)
        scale = (b.abs().amax((1, 3), keepdim=True) / TOP).float()
        inv = (1 / scale.double()).float().double()
        there = scale >= 2.0 ** -126
        q = (b * inv).float().double()
        y = torch.where(there, _e4m3(torch.where(there, q, 0.0)) * scale.double(), 0.0)
        out[lo : lo + tall] = y.reshape(full.shape)[:t, :K]
    return out


def _weights(s):
    """The weights' values: each code times its block's scale."""
    N, K = s["w"].shape
    o, k = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    return s["w"].double() * s["ws"].double()[o][:, k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        y = _block_values(s["x"].double(), 1, 128) @ _weights(s).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "product_gradients":
        dy, x = s["dy"].double(), s["x"].double()
        return {"X": _block_values(dy, 1, 128) @ _weights(s), "W": _block_values(dy, 128, 1).t() @ _block_values(x, 128, 1)}
    if op.startswith("heads"):
        T, R = case["T"], case["R"]
        turn = torch.polar(torch.ones((T, 1, R // 2), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), s["freqs"])[:, None])

        def forward(x, w):
            n = x / (x.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w
            r = n[..., :R]
            if case["pairs"] == "halves":
                z = torch.complex(r[..., : R // 2], r[..., R // 2 :]) * turn
                r = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.complex(r[..., ::2], r[..., 1::2]) * turn
                r = torch.view_as_real(z).flatten(-2)
            return torch.cat([r, n[..., R:]], -1)

        q, k, qw, kw = (s[n].double().requires_grad_() for n in ("q", "k", "qw", "kw"))
        yq, yk = forward(q, qw), forward(k, kw)
        if op == "heads":
            return [yq.detach(), yk.detach()]
        dq, dqw = torch.autograd.grad(yq, [q, qw], s["dq"].double())
        dk, dkw = torch.autograd.grad(yk, [k, kw], s["dk"].double())
        return {"Q": dq, "K": dk, "q_weight": dqw, "k_weight": dkw}
    return _adamw_exact(s)


def _adamw_exact(s):
    f, a = s["flat"], s["args"]
    (b1, b2), t = a["betas"], a["step"]
    eight = s["case"]["bits"] == 8
    out = {k: torch.zeros(x.shape, dtype=torch.float64, device="cuda") for k, x in f.items() if k != "g"}
    for i, (lo, n) in enumerate(zip(*s["place"])):
        each = 1 << 24
        for a0 in range(0, n, each):  # in pieces of whole groups
            hi = min(n, a0 + each)
            at, place = slice(lo + a0, lo + hi), torch.arange(a0, hi, device="cuda")
            g = f["g"][at].double() * a["grad_scale"]
            m, v = f["m"][at].double(), f["v"][at].double()
            group = (lo + place) // GROUP
            if eight:
                m, v = m * f["m_scales"].double()[group], (v * f["v_scales"].double()[group]) ** 2
            m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
            step = (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + a["eps"])
            p = f["p"][at].double()
            p = p - a["lr"] * (step + a["weight_decay"] * p)
            out["p"][at] = p
            if "copy" in f:
                out["copy"][at] = p
            if not eight:
                out["m"][at], out["v"][at] = m, v
                continue
            h = _bits(place, s["seed"], t, i)
            for name, x, bits in (("m", m, h >> 16), ("v", v.sqrt(), h & 0xFFFF)):
                first = group - group[0]
                top = torch.zeros(int(first[-1]) + 1, dtype=torch.float64, device="cuda")
                top.scatter_reduce_(0, first, x.abs(), "amax")
                scale = top / TOP
                q = x.abs() / scale.clamp(min=1e-300)[first]
                unit = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
                code = (torch.floor(q / unit + bits / 65536.0) * unit).clamp(max=TOP)
                if name == "v":
                    code = torch.where((q > 0) & (code == 0), 2.0 ** -9, code)
                out[name][at] = code * x.sign()
                out[name + "_scales"][group[0] : group[-1] + 1] = scale
    return out
