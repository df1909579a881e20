"""The AdamW step over many tensors (bakron_adamw), against fp64.

In units of E = 2^-24.  The constants are rounded once.  A new moment is off by
4 (|b1 m| + |c1 g|), a new square by 6 of itself (all terms positive); the root
by half of that and 2 for the approximate square root; the divisor by 2 more,
its reciprocal by 2, and the step's product with them by 3: 16 of the step, and
the moment's own error through the same factor.  The parameter takes 3
roundings of its own size, and that of its type, u (2^-24, 2^-11, 2^-8; fp16
adds half its smallest step, 2^-25).

8-bit states are cut at random: up where the 16 random bits, as a fraction of
a step, reach beyond what is cut off.  That is monotone in the value, so a code
lies between those of values 48 E smaller and larger (the moment's error, the
scale's and the quotient's), given the same bits."""

import math

import numpy as np
import pytest

from test_gpu_int8_matmul import U, bk  # noqa: F401

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
GROUP = 256


def _bits(i, seed, step, place):
    """32 random bits of the value at i of the tensor at `place` of the list."""
    m = 0xFFFFFFFF
    x = (i * 0x9E3779B1 + (i >> 32) * 0xBB67AE85 + ((seed * 0x9E3779B1 + step * 0x6A09E667 + place * 0xBB67AE85) & m)) & m
    x = ((x ^ (x >> 16)) * 0x6A09E667) & m
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & m
    return x ^ (x >> 16)


def _cut(q, bits):
    """The number of e4m3 that q >= 0 is cut to."""
    import torch

    unit = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
    return (torch.floor(q / unit + bits.double() / 65536) * unit).clamp(max=448.0)


def _make(rng, sizes, dtype, grad, bits, first=False):
    import torch

    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    params = [cuda(0.05 * rng.standard_normal(n)).to(getattr(torch, dtype)) for n in sizes]
    spread = [np.exp(rng.standard_normal(n)) for n in sizes]
    grads = [cuda(1e-2 * s * rng.standard_normal(n)).to(getattr(torch, grad)) for n, s in zip(sizes, spread)]
    m = [cuda(3e-3 * s * rng.standard_normal(n)) for n, s in zip(sizes, spread)]
    v = [cuda(1e-4 * s * s * rng.uniform(0.5, 2, n)) for n, s in zip(sizes, spread)]
    if first:
        m, v = [torch.zeros_like(x) for x in m], [torch.zeros_like(x) for x in v]
    if bits == 32:
        return params, grads, {"m": m, "v": v}
    states = {"m": [], "v": [], "m_scales": [], "v_scales": []}
    for name, xs in (("m", m), ("v", [x.sqrt() for x in v])):
        for x in xs:
            n = len(x)
            full = torch.zeros(-(-n // GROUP) * GROUP, device="cuda")
            full[:n] = x
            scale = full.view(-1, GROUP).abs().amax(1) / 448
            q = (full.view(-1, GROUP) / scale.clamp(min=1e-38)[:, None]).clamp(-448, 448)
            states[name].append(q.to(torch.float8_e4m3fn).view(-1)[:n].clone())
            states[name + "_scales"].append(scale)
    return params, grads, states


ARGS = {"step": 7, "lr": 3e-3, "betas": (0.9, 0.99), "eps": 1e-7, "weight_decay": 0.05, "grad_scale": 0.25}


def _copy(states):
    return {k: [t.clone() for t in l] for k, l in states.items()}


def _check(before, grads, old, params, states, copies, args, seed=0, places=None):
    """One step from (before, old) in fp64 against (params, states)."""
    import torch

    (b1, b2), t, lr = args["betas"], args["step"], args["lr"]
    eight = "m_scales" in old
    for i, (p0, g) in enumerate(zip(before, grads)):
        n = p0.numel()
        if n == 0:
            continue
        g = g.double().flatten() * args["grad_scale"]
        m0, v0 = old["m"][i].double(), old["v"][i].double()
        group = torch.arange(n, device="cuda") // GROUP
        if eight:
            m0, v0 = m0 * old["m_scales"][i].double()[group], (v0 * old["v_scales"][i].double()[group]) ** 2
        m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        em = 4 * E * (b1 * m0.abs() + (1 - b1) * g.abs()) + 1e-44
        d = v.sqrt() / math.sqrt(1 - b2 ** t) + args["eps"]
        rate = lr / (1 - b1 ** t)
        step = torch.where(m == 0, 0.0, rate * m / d)
        p = p0.double().flatten()
        want = p * (1 - lr * args["weight_decay"]) - step
        off = rate * em / d + 16 * E * step.abs() + 3 * E * p.abs()
        for out, kind in ((params[i], p0.dtype), (copies[i], copies[i].dtype) if copies and copies[i] is not None else (None, None)):
            if out is None:
                continue
            name = str(kind).replace("torch.", "")
            tol = off + U[name] * want.abs() * (1 + 2.0 ** -8) + (2.0 ** -25 if name == "float16" else 1e-40)
            bad = ((out.double().flatten() - want).abs() / tol).max()
            assert float(bad) <= 1.0, (i, name, float(bad))
        if not eight:
            assert bool(((states["m"][i].double() - m).abs() <= em).all())
            assert bool(((states["v"][i].double() - v).abs() <= 6 * E * v + 1e-44).all())
            continue
        h = _bits(torch.arange(n, device="cuda"), seed, t, i)
        for name, x, bits in (("m", m, h >> 16), ("v", v.sqrt(), h & 0xFFFF)):
            top = torch.zeros(-(-n // GROUP), dtype=torch.float64, device="cuda").scatter_reduce_(0, group, x.abs(), "amax")
            got = states[name + "_scales"][i].double()
            assert bool(((got - top / 448).abs() <= 16 * E * top / 448 + 1e-44).all())
            scale = torch.where(got > 0, got, 1.0)[group]
            ex = (em if name == "m" else 8 * E * x) + 48 * E * x.abs()
            lo, hi = ((x.abs() - ex).clamp(min=0) / scale).clamp(max=448), ((x.abs() + ex) / scale).clamp(max=448)
            lo, hi = _cut(lo, bits), _cut(hi, bits)
            if name == "v":  # what is not 0 stays so
                lo, hi = torch.where(x > 0, lo.clamp(min=2.0 ** -9), 0), torch.where(x > 0, hi.clamp(min=2.0 ** -9), 0)
            code = states[name][i].double()
            assert bool(((code.abs() >= lo) & (code.abs() <= hi))[got[group] > 0].all()), (i, name)
            assert not code[got[group] == 0].any()
            assert bool((code * x.sign() >= 0)[x.abs() > ex].all())


SIZES = [[1], [255, 256, 257], [64, 0, 5, 100003], list(range(1, 140)), [2048, 4096, 70000, 3]]


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype,grad", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                        ("bfloat16", "float32"), ("float16", "float16")])
@pytest.mark.parametrize("sizes", SIZES, ids=len)
def test_step(bk, sizes, dtype, grad, bits):  # noqa: F811
    import torch

    rng = np.random.default_rng(len(sizes) + bits)
    params, grads, states = _make(rng, sizes, dtype, grad, bits)
    copies = [p.to(torch.bfloat16 if i % 2 else torch.float16, copy=True) if i % 3 else None for i, p in enumerate(params)]
    before, old, keep = [p.clone() for p in params], _copy(states), [g.clone() for g in grads]
    st = bk.adamw(params, grads, states, copies=copies, seed=5, **ARGS)
    assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(grads, keep))
    _check(before, grads, old, params, states, copies, ARGS, seed=5)


@pytest.mark.parametrize("bits", [8, 32])
def test_first_steps_from_nothing(bk, bits):  # noqa: F811
    """States of adamw_states, two steps with gradients of other sizes, matrices as parameters, zeros among the gradients."""
    import torch

    rng = np.random.default_rng(3)
    params = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in ((30, 50), (7,), (2, 3, 300))]
    states = bk.adamw_states(params, bits)
    for step in (1, 2):
        grads = [torch.from_numpy((10.0 ** (-3 * step) * rng.standard_normal(p.shape)).astype(np.float32)).cuda() for p in params]
        grads[0][3:20] = 0
        before, old = [p.clone() for p in params], _copy(states)
        args = {**ARGS, "step": step}
        assert int(bk.adamw(params, grads, states, **args).item()) == 0
        _check(before, grads, old, params, states, None, args)


@pytest.mark.parametrize("bits", [8, 32])
def test_unaligned_tensors_and_neighbours_left_alone(bk, bits):  # noqa: F811
    """Parameters, gradients and states at odd places of larger buffers, whose other values stay what they were."""
    import torch

    rng = np.random.default_rng(4)
    sizes = [300, 1000, 5, 257]
    params, grads, states = _make(rng, sizes, "bfloat16", "float32", bits)
    before, old = [p.clone() for p in params], _copy(states)

    def placed(ts, mark):
        room, out, at = [], [], []
        for i, t in enumerate(ts):
            r = torch.full((len(t) + 8 + i,), mark, device="cuda").to(t.dtype)
            a = 1 + i
            r[a : a + len(t)] = t
            room.append(r), out.append(r[a : a + len(t)]), at.append(a)
        return room, out, at

    rooms = {}
    rooms["p"], params, _ = placed(params, 3.0)
    _, grads, _ = placed(grads, 3.0)
    for k in states:
        rooms[k], states[k], _ = placed(states[k], 3.0)
    bk.adamw(params, grads, states, seed=9, **ARGS)
    _check(before, grads, old, params, states, None, ARGS, seed=9)
    for room in rooms.values():
        for i, r in enumerate(room):
            assert bool((r[: 1 + i].float() == 3).all()) and bool((r[-7:].float() == 3).all())


def test_the_same_step_in_any_alignment_and_company(bk):  # noqa: F811
    """Alone, a tensor at the first place of the list gives what it gives among others."""
    import torch

    rng = np.random.default_rng(5)
    for bits in (8, 32):
        params, grads, states = _make(rng, [5000, 300, 7], "float32", "bfloat16", bits)
        alone = [params[0].clone()], [grads[0]], {k: [l[0].clone()] for k, l in states.items()}
        odd = torch.empty(5001, device="cuda")[1:].copy_(params[0])
        other = [odd], [grads[0]], {k: [l[0].clone()] for k, l in states.items()}
        for p, g, s in ((params, grads, states), alone, other):
            bk.adamw(p, g, s, seed=3, **ARGS)
        for p, _, s in (alone, other):
            assert torch.equal(p[0], params[0])
            assert all(torch.equal(s[k][0].view(torch.uint8), states[k][0].view(torch.uint8)) for k in s)


@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_a_launch_takes(bk, bits):  # noqa: F811
    import torch

    rng = np.random.default_rng(11)
    sizes = [int(n) for n in rng.integers(0, 600, 801)]
    params, grads, states = _make(rng, sizes, "float32", "bfloat16", bits)
    before, old = [p.clone() for p in params], _copy(states)
    assert int(bk.adamw(params, grads, states, seed=4, **ARGS).item()) == 0
    _check(before, grads, old, params, states, None, ARGS, seed=4)


def test_the_same_tensor_twice(bk):  # noqa: F811
    """Two steps of one parameter, or of one state, at once would race: refused, and nothing changes."""
    import torch

    params, grads, states = _make(np.random.default_rng(12), [300, 300], "float32", "float32", 32)
    before = [p.clone() for p in params]
    twice = {"m": [states["m"][0]] * 2, "v": states["v"]}
    for p, s, c in (([params[0]] * 2, states, None), (params, twice, None), (params, states, [params[0].half()] * 2)):
        with pytest.raises(RuntimeError):
            bk.adamw(p, grads, s, copies=c, **ARGS)
    assert all(torch.equal(a, b) for a, b in zip(params, before))


def test_rounding_at_random_is_without_bias(bk):  # noqa: F811
    """Values between two codes, over many seeds: the mean is the value, within 6 standard deviations of the mean."""
    import torch

    n, seeds = 4096, 400
    q = torch.linspace(0.0005, 440, n, device="cuda")
    q[::256] = 448
    m = q / 448 * 1e-2
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    states = bk.adamw_states([p])
    for k in ("m", "m_scales", "v", "v_scales"):
        assert k in bk.adamw_states([p], 8)
    # m as a gradient with beta1 = 0, so that the new moment is the gradient itself
    g.copy_(m)
    for seed in range(seeds):
        states = bk.adamw_states([p], 8)
        bk.adamw([p], [g], states, 1, lr=0.0, betas=(0.0, 0.9), weight_decay=0.0, seed=seed)
        total += states["m"][0].double() * states["m_scales"][0].double().repeat_interleave(GROUP)
    exact = m.double()
    unit = torch.exp2(torch.floor(torch.log2((exact / exact.view(-1, GROUP).amax(1).repeat_interleave(GROUP) * 448).clamp(min=2.0 ** -6))) - 3)
    unit = unit * exact.view(-1, GROUP).amax(1).repeat_interleave(GROUP) / 448
    assert bool(((total / seeds - exact).abs() <= 6 * 0.5 * unit / math.sqrt(seeds) + 1e-6 * exact + 2.0 ** -16 * unit).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_that_are_not_finite(bk, bits):  # noqa: F811
    """Such a value and its states stay, and the status says so; so does one whose square overflows."""
    import torch

    rng = np.random.default_rng(6)
    params, grads, states = _make(rng, [700, 300], "float32", "float32", bits)
    clean_p, clean_s = [p.clone() for p in params], _copy(states)
    before, old = [p.clone() for p in params], _copy(states)
    bad = [3, 255, 256, 699]
    quiet = [g.clone() for g in grads]
    for i, x in zip(bad, (float("nan"), float("inf"), -float("inf"), 3e38)):
        grads[0][i] = x
    st = bk.adamw(params, grads, states, seed=1, **ARGS)
    assert int(st.item()) == bk._lib.DEV_NONFINITE_GRAD
    assert int(bk.adamw(clean_p, quiet, clean_s, seed=1, **ARGS).item()) == 0
    others = torch.ones(700, dtype=torch.bool, device="cuda")
    others[bad] = False
    assert torch.equal(params[0][bad], before[0][bad]) and torch.equal(params[0][others], clean_p[0][others])
    assert torch.equal(params[1], clean_p[1])
    if bits == 32:
        assert all(torch.equal(states[k][0][bad], old[k][0][bad]) for k in "mv")
        assert all(torch.equal(states[k][0][others], clean_s[k][0][others]) for k in "mv")
    else:
        assert all(bool(torch.isfinite(states[k][0].float()).all()) for k in ("m", "v", "m_scales", "v_scales"))
        for k in "mv":  # rounded again, by one step at most
            a, b = states[k][0][bad].float() * states[k + "_scales"][0][torch.tensor(bad) // GROUP], \
                old[k][0][bad].float() * old[k + "_scales"][0][torch.tensor(bad) // GROUP]
            step = torch.maximum(b.abs() * 2.0 ** -3, states[k + "_scales"][0][torch.tensor(bad) // GROUP] * 2.0 ** -9)
            assert bool(((a - b).abs() <= step * 1.01).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_numbers_on_the_device_and_skipped_steps(bk, bits):  # noqa: F811
    import torch

    rng = np.random.default_rng(7)
    params, grads, states = _make(rng, [5000, 33], "float32", "bfloat16", bits)
    other, old = [p.clone() for p in params], _copy(states)
    dev = {"step": torch.tensor(7, device="cuda"), "lr": torch.tensor([3e-3], device="cuda"),
           "grad_scale": torch.tensor(0.25, device="cuda")}
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    args = {**ARGS, **dev}
    before = [p.clone() for p in params]
    bk.adamw(params, grads, states, skip=skip, **args)
    assert all(torch.equal(a, b) for a, b in zip(params, before))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for k in states for a, b in zip(states[k], old[k]))
    skip.zero_()
    bk.adamw(params, grads, states, skip=skip, **args)
    # lr as a float32 number: so is the host's
    bk.adamw(other, grads, old, **{**ARGS, "lr": float(np.float32(3e-3))})
    assert all(torch.equal(a, b) for a, b in zip(params, other))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for k in states for a, b in zip(states[k], old[k]))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_and_replayed(bk, bits):  # noqa: F811
    """A step that a graph replays, with its number counted on the device, is the step of a call by itself."""
    import torch

    rng = np.random.default_rng(8)
    params, grads, states = _make(rng, [70000] + [300] * 200, "float32", "bfloat16", bits)
    other, mine = [p.clone() for p in params], _copy(states)
    step, skip = torch.full((1,), 10, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = {k: v for k, v in ARGS.items() if k != "step"}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step += 1
        status = bk.adamw(params, grads, states, step, skip=skip, **args)
    for turn in range(3):
        for g in grads:
            g.mul_(-0.7)
        graph.replay()
        alone = bk.adamw(other, grads, mine, 11 + turn, **args)
        assert int(status.item()) == int(alone.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(params, other))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for k in states for a, b in zip(states[k], mine[k]))


def test_another_stream(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(9)
    params, grads, states = _make(rng, [5000, 12], "float32", "float32", 8)
    other, mine = [p.clone() for p in params], _copy(states)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st = bk.adamw(params, grads, states, stream=side, **ARGS)
    torch.cuda.current_stream().wait_stream(side)
    bk.adamw(other, grads, mine, **ARGS)
    assert int(st.item()) == 0 and all(torch.equal(a, b) for a, b in zip(params, other))


def test_places_beyond_32_bits(bk):  # noqa: F811
    """The last values of a tensor of more than 2^32 values (8.6 GB of parameters, 8-bit states), step for step."""
    import torch

    n = (1 << 32) + 517
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = slice((1 << 32) - 256, n)
    rng = np.random.default_rng(10)
    m = n - tail.start
    p[tail], g[tail] = (torch.from_numpy(rng.standard_normal(m).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    states = bk.adamw_states([p], 8)
    before = p[tail].clone()
    assert int(bk.adamw([p], [g], states, seed=2, **ARGS).item()) == 0
    want = [before.clone()]
    small = bk.adamw_states(want, 8)
    bk.adamw(want, [g[tail].clone()], small, seed=2, **ARGS)
    assert torch.equal(p[tail], want[0])
    assert torch.equal(states["m_scales"][0][tail.start // GROUP :], small["m_scales"][0])
    x = g[tail].double() * ARGS["grad_scale"] * 0.1
    h = _bits(torch.arange(tail.start, n, device="cuda"), 2, ARGS["step"], 0)
    scale = small["m_scales"][0].double()[torch.arange(m, device="cuda") // GROUP]
    lo, hi = ((x.abs() * (1 + s * 48 * E) / scale).clamp(max=448) for s in (-1, 1))
    code = states["m"][0][tail].double().abs()
    assert bool(((code >= _cut(lo, h >> 16)) & (code <= _cut(hi, h >> 16))).all())


def test_refusals(bk):  # noqa: F811
    import torch

    p, g = [torch.ones(300, device="cuda")], [torch.ones(300, device="cuda")]
    s32, s8 = bk.adamw_states(p), bk.adamw_states(p, 8)
    one = torch.ones(1, device="cuda")
    for call in (lambda: bk.adamw([], [], {"m": [], "v": []}, 1), lambda: bk.adamw([p[0].cpu()], g, s32, 1), lambda: bk.adamw(p, [], s32, 1),
                 lambda: bk.adamw(p, [g[0][:200]], s32, 1), lambda: bk.adamw(p, [g[0].double()], s32, 1),
                 lambda: bk.adamw(p, [g[0].cpu()], s32, 1), lambda: bk.adamw([torch.ones((2, 600), device="cuda")[:, ::2]], [torch.ones(600, device="cuda")], bk.adamw_states([torch.ones(600, device="cuda")]), 1),
                 lambda: bk.adamw(p, g, {"m": s32["m"], "v": [one]}, 1), lambda: bk.adamw(p, g, {**s8, "v_scales": [one]}, 1),
                 lambda: bk.adamw(p, g, {**s32, "m_scales": s8["m_scales"], "v_scales": s8["v_scales"]}, 1),
                 lambda: bk.adamw(p, g, s32, 0), lambda: bk.adamw(p, g, s32, one), lambda: bk.adamw(p, g, s32, 1, lr=one.double()),
                 lambda: bk.adamw(p, g, s32, 1, skip=1), lambda: bk.adamw(p, g, s32, 1, skip=one),
                 lambda: bk.adamw(p, g, s32, 1, copies=[one.half()]), lambda: bk.adamw(p, g, s32, 1, copies=[p[0]]),
                 lambda: bk.adamw(p, g, s32, 1, copies=[]), lambda: bk.adamw_states(p, 16)):
        with pytest.raises(ValueError):
            call()
    for bad in ({"betas": (1.0, 0.9)}, {"betas": (0.9, -0.1)}, {"eps": -1.0}, {"lr": float("nan")}):
        with pytest.raises(RuntimeError):
            bk.adamw(p, g, s32, 1, **bad)
    with pytest.raises(RuntimeError):  # the parameter as its own gradient
        bk.adamw(p, p, s32, 1)
    assert bool((p[0] == 1).all())


def test_codes_are_those_of_elementary_operations(bk):  # noqa: F811
    """Four million values against torch's fp32 products, sums, root and quotients, each rounded by itself.  At most one
    root in 10^5 is a neighbour of the nearest number, and a cut notices a last place in one of 10^5 at most (16 steps of
    2^-24 of a value): fewer than one code here, and four scales."""
    import torch

    n = 1 << 22
    gen = torch.Generator("cuda").manual_seed(3)
    rand = lambda: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    p, g = [0.02 * rand()], [(1e-3 * torch.exp(rand()) * rand()).bfloat16()]
    states = bk.adamw_states(p, 8)
    (b1, b2), t = ARGS["betas"], ARGS["step"]
    for turn in range(2):
        m = states["m"][0].float().view(-1, GROUP) * states["m_scales"][0][:, None]
        v = (states["v"][0].float().view(-1, GROUP) * states["v_scales"][0][:, None]).square()
        x = g[0].float().view(-1, GROUP) * ARGS["grad_scale"]
        m = m * b1 + x * (1 - b1)
        root = (v * b2 + x * x * (1 - b2)).sqrt()
        bk.adamw(p, g, states, seed=turn, **ARGS)
        bits = _bits(torch.arange(n, device="cuda"), turn, t, 0).view(-1, GROUP)
        for name, y, b in (("m", m, bits >> 16), ("v", root, bits & 0xFFFF)):
            top = y.abs().amax(1)
            scale = top / torch.full_like(top, 448.0)
            q = (y.abs() * (1 / scale)[:, None])
            u = q.view(torch.int32)
            code = torch.where(q >= 2.0 ** -6, ((u + (b.int() << 4)) >> 20) - 960, (q * 512 + b.float() * 2.0 ** -16).int()).clamp(max=126)
            code = torch.where((q > 0) & (code == 0), 1, code) if name == "v" else code
            got = states[name][0].view(torch.uint8).view(-1, GROUP)
            assert int((states[name + "_scales"][0] != scale).sum()) <= 4
            assert int(((got & 127) != code).sum()) <= 4
        g[0].mul_(-0.5)
