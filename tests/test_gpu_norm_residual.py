"""The norms around a block with its gate and residual sum
(bakron_norm_residual) and their gradients, against fp64.

Tolerance: a row sum of D terms passes through at most 32 additions in a
thread, ten in the shuffles and eight across a cluster, and a value through a
dozen more roundings, so every fp32 result is within c 2^-24 of the sum of the
magnitudes of what was added to make it, c = 64 for each sum on the way (at
most four: mean, deviation, and the same of the next norm or gradient); 256 in
all.  The references below carry those magnitudes along (the same formulas
with absolute values).  A sum over tokens adds the number of tokens to c.
Results in 16 bits add their own rounding, 2^-11 or 2^-8 (fp16: and 2^-25).
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
C = 256 * 2.0 ** -24
EPS, ALPHA = 1e-5, 0.75


@pytest.fixture(scope="module")
def bk():
    import torch

    import kronecker_hessian_gptq_gb300 as bk
    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    bk.load_library()
    torch.cuda.init()
    return bk


def _make(t, d, dtype, kind, groups, post=True, pre=True, seed=0):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed + 31 * t + d)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    to = getattr(torch, dtype)
    a = {"post": 1 + 0.2 * rand(d) if post else None, "pre": 1 + 0.2 * rand(d) if pre else None,
         "gate": (0.5 * rand(groups, d)).to(to) if groups else None}
    layer = kind == "layer"
    a["post_bias"] = 0.3 * rand(d) if layer and post else None
    a["pre_bias"] = 0.3 * rand(d) if layer and pre else None
    x, h, dy, dz = ((rand(t, d) + 0.5).to(to) for _ in range(4))
    return x, h, dy, dz, a


def _norm(v, mag, w, b, kind):
    """(values, magnitudes, unit rows, their magnitudes, 1 / deviation) of a norm in fp64; mag: v's magnitudes."""
    m = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    mm = mag + mag.mean(1, keepdim=True) if kind == "layer" else mag
    r = ((v - m).pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    n = (v - m) * r
    # an error of the row moves the deviation too, by at most its rms
    nm = (mm + n.abs() * mm.pow(2).mean(1, keepdim=True).sqrt()) * r + n.abs()
    out, om = n, nm
    if w is not None:
        out, om = out * w.double(), om * w.double().abs()
    if b is not None:
        out, om = out + b.double(), om + b.double().abs()
    return out, om, n, nm, r


def _gate(a, t):
    import torch

    return 1.0 if a["gate"] is None else torch.repeat_interleave(a["gate"].double(), t // a["gate"].shape[0], 0)


def _forward(x, h, a, kind):
    x = ALPHA * x.double()
    y, ym = x, x.abs()
    if h is not None:
        u = um = None
        if a["post"] is None:
            u, um = h.double(), h.double().abs()
        else:
            u, um = _norm(h.double(), h.double().abs(), a["post"], a["post_bias"], kind)[:2]
        g = _gate(a, len(x))
        y, ym = y + g * u, ym + (g.abs() * um if a["gate"] is not None else um)
    z = zm = None
    if a["pre"] is not None:
        z, zm = _norm(y, ym, a["pre"], a["pre_bias"], kind)[:2]
    return y, ym, z, zm


def _within(got, ref, mag, dtype, c=C):
    import torch

    tol = c * mag + U[dtype] * ref.abs() * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == "float16" else 1e-30)
    worst = float(((got.double() - ref).abs() / tol).max())
    assert torch.isfinite(got).all() and worst <= 1.0, worst


SHAPES = [(1, 1), (1, 4096), (3, 5), (7, 64), (33, 1000), (5, 1999), (16, 8192), (9, 8200), (4, 14336), (2, 20000), (3, 32768),
          (130, 264), (12, 4100), (2, 32765)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,d", SHAPES)
def test_forward(bk, t, d, dtype, kind):
    for groups in sorted({0, 1, t}):
        x, h, _, _, a = _make(t, d, dtype, kind, groups)
        y, z = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
        ry, ym, rz, zm = _forward(x, h, a, kind)
        _within(y, ry, ym, dtype)
        _within(z, rz, zm, dtype)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,pre,block", [(True, False, True), (False, True, True), (False, False, True), (False, True, False)])
def test_forward_with_parts_left_out(bk, kind, post, pre, block):
    for t, d in ((6, 520), (5, 77)):
        x, h, _, _, a = _make(t, d, "bfloat16", kind, 2 if block and t % 2 == 0 else 0, post, pre)
        h = h if block else None
        y, z = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
        ry, ym, rz, zm = _forward(x, h, a, kind)
        _within(y, ry, ym, "bfloat16")
        if pre:
            _within(z, rz, zm, "bfloat16")
        else:
            assert z is None


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("t,d", [(1, 4096), (7, 129), (20, 1000), (3, 14336), (2, 20000)])
def test_codes_of_the_norm(bk, t, d, dtype, kind):
    """Codes times scale are within half a step of the norm, and the scale is the largest magnitude / 127."""
    x, h, _, _, a = _make(t, d, dtype, kind, 1)
    y, c, s = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind, codes=True)
    y2, _ = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    ry, ym, rz, zm = _forward(x, h, a, kind)
    assert (y == y2).all()
    top = rz.abs().amax(1)
    err = (C * zm).amax(1)
    assert bool(((s.double() * 127 - top).abs() <= err + 2.0 ** -23 * top).all())
    assert bool(((c.double() * s.double()[:, None] - rz).abs() <= 0.5 * s.double()[:, None] * (1 + 1e-4) + C * zm).all())
    assert int(c.abs().max()) == 127 and bool((c.abs().amax(1) == 127).all())


def _reference_gradients(dy, dz, y, h, a, kind):
    t = len(y)
    dt, dtm = (0.0, 0.0) if dy is None else (dy.double(), dy.double().abs())
    out = {}
    if dz is not None:
        y = y.double()
        _, _, n, nm, r = _norm(y, y.abs(), None, None, kind)
        k = dz.double() * a["pre"].double()
        dt = dt + r * (k - (k.mean(1, keepdim=True) if kind == "layer" else 0) - n * (k * n).mean(1, keepdim=True))
        km = k.abs()
        dtm = dtm + r * (km + (km.mean(1, keepdim=True) if kind == "layer" else 0) + nm * (km * nm).mean(1, keepdim=True))
        out["pre"] = ((dz.double() * n).sum(0), (dz.double().abs() * nm).sum(0))
        out["pre_bias"] = (dz.double().sum(0), dz.double().abs().sum(0))
    out["X"] = (ALPHA * dt, ALPHA * dtm)
    if h is None:
        return out
    h = h.double()
    g = _gate(a, t)
    gm = g.abs() if a["gate"] is not None else 1.0
    du, dum = dt * g, dtm * gm
    if a["post"] is None:
        u, um, dh, dhm = h, h.abs(), du, dum
    else:
        u, um, n, nm, r = _norm(h, h.abs(), a["post"], a["post_bias"], kind)
        q, qm = du * a["post"].double(), dum * a["post"].double().abs()
        dh = r * (q - (q.mean(1, keepdim=True) if kind == "layer" else 0) - n * (q * n).mean(1, keepdim=True))
        dhm = r * (qm + (qm.mean(1, keepdim=True) if kind == "layer" else 0) + nm * (qm * nm).mean(1, keepdim=True))
        out["post"] = ((du * n).sum(0), (dum * nm).sum(0))
        out["post_bias"] = (du.sum(0), dum.sum(0))
    out["H"] = (dh, dhm)
    if a["gate"] is not None:
        groups, d = a["gate"].shape
        out["gate"] = tuple(v.view(groups, t // groups, d).sum(1) for v in (dt * u, dtm * um))
    return out


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,d,groups", [(1, 1, 1), (1, 4096, 0), (1, 4096, 1), (3, 5, 3), (7, 64, 1), (350, 264, 1), (350, 264, 7),
                                        (700, 72, 700), (660, 40, 330), (33, 1000, 11), (5, 1999, 1), (16, 8192, 2),
                                        (9, 8200, 3), (4, 14336, 2), (2, 20000, 1), (3, 32768, 3), (4, 32765, 1)])
def test_backward(bk, t, d, groups, dtype, kind):
    y, h, dy, dz, a = _make(t, d, dtype, kind, groups)
    got = bk.norm_residual_backward(dy, dz, y, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    ref = _reference_gradients(dy, dz, y, h, a, kind)
    for name, value in got.items():
        if kind == "rms" and name.endswith("bias") or (name == "gate" and not groups):
            assert value is None
            continue
        full = name in ("X", "H")
        _within(value, *ref[name], dtype if full else "float32", C if full else C + t * 2.0 ** -24)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,use_dy,use_dz,block", [(False, True, True, True), (True, True, False, True),
                                                      (True, False, True, True), (False, True, True, False)])
def test_backward_with_parts_left_out(bk, kind, post, use_dy, use_dz, block):
    for t, d in ((6, 520), (5, 77)):
        y, h, dy, dz, a = _make(t, d, "float32", kind, 1 if block else 0, post and block, use_dz)
        h, dy, dz = h if block else None, dy if use_dy else None, dz if use_dz else None
        got = bk.norm_residual_backward(dy, dz, y, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
        ref = _reference_gradients(dy, dz, y, h, a, kind)
        for name, value in got.items():
            if value is not None:
                _within(value, *ref[name], "float32", C + t * 2.0 ** -24)
        assert {k for k, v in got.items() if v is not None} == {k for k in ref if kind == "layer" or "bias" not in k}


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(bk, kind):
    """Central differences of the fp64 forward along random directions, one input at a time.

    The step 1e-5 leaves about 1e-9 of truncation; the gradients themselves are within the bound above."""
    import torch

    t, d = 12, 96
    x, h, dy, dz, a = _make(t, d, "float32", kind, 3)
    y64 = _forward(x, h, a, kind)[0]
    y = y64.float()
    got = bk.norm_residual_backward(dy, dz, y, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    ref = _reference_gradients(dy, dz, y, h, a, kind)

    def value(x, h, a):
        ry, _, rz, _ = _forward(x, h, a, kind)
        return float((ry * dy.double()).sum() + (rz * dz.double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(9)
    for name, at in [("X", x), ("H", h)] + [(k, v) for k, v in a.items() if v is not None]:
        step = torch.randn(at.shape, generator=gen, device="cuda", dtype=torch.float64)
        moved = []
        for sign in (1, -1):
            new = at.double() + sign * 1e-5 * step
            moved.append(value(new if name == "X" else x, new if name == "H" else h, {**a, **({name: new} if name in a else {})}))
        slope = (moved[0] - moved[1]) / 2e-5
        tol = float((step.abs() * ((C + t * 2.0 ** -24) * ref[name][1] + 2.0 ** -23 * ref[name][0].abs())).sum())
        # y is rounded to fp32 before the gradients are taken: 2^-24 of what they depend on it through, far within C
        assert abs(float((got[name].double() * step).sum()) - slope) <= tol + 1e-6 * abs(slope) + 1e-6


def test_strides_alignment_and_in_place_sums(bk):
    import torch

    for d, off in ((256, 8), (256, 1), (250, 3)):
        x, h, dy, dz, a = _make(10, 300, "bfloat16", "rms", 2)
        cut = lambda v: None if v is None else v[..., off : off + d]  # noqa: E731
        b = {k: None if v is None else cut(v).contiguous() if k != "gate" else cut(v) for k, v in a.items()}
        strided = bk.norm_residual(cut(x), cut(h), **b)
        dense = bk.norm_residual(cut(x).contiguous(), cut(h).contiguous(), **{**b, "gate": b["gate"].contiguous()})
        assert all(torch.equal(p, q) for p, q in zip(strided, dense))
        gs = bk.norm_residual_backward(cut(dy), cut(dz), cut(x), cut(h), **b)
        gd = bk.norm_residual_backward(*(cut(v).contiguous() for v in (dy, dz, x, h)), **{**b, "gate": b["gate"].contiguous()})
        for k in gs:
            assert (gs[k] is None and gd[k] is None) or torch.allclose(gs[k].float(), gd[k].float(), rtol=2.0 ** -7, atol=1e-5), k


def test_values_that_are_not_finite_stay_in_their_row(bk):
    import torch

    x, h, dy, dz, a = _make(20, 256, "bfloat16", "layer", 4)
    clean = bk.norm_residual(x, h, **a, kind="layer")
    h[7, 3] = float("nan")
    x[11, 200] = float("inf")
    y, z = bk.norm_residual(x, h, **a, kind="layer")
    rest = [i for i in range(20) if i not in (7, 11)]
    assert torch.equal(y[rest], clean[0][rest]) and torch.equal(z[rest], clean[1][rest])
    assert torch.isnan(z[7]).all() and torch.isnan(z[11]).all()
    _, c, s = bk.norm_residual(x, h, **a, kind="layer", codes=True)
    assert torch.isnan(s[[7, 11]]).all() and torch.isfinite(s[rest]).all() and not c[[7, 11]].any()


def test_rows_of_zeros(bk):
    import torch

    z = torch.zeros((3, 512), device="cuda", dtype=torch.float16)
    w = torch.ones(512, device="cuda")
    y, c, s = bk.norm_residual(z, z, post=w, pre=w, codes=True)
    assert not y.any() and not c.any() and not s.any()
    g = bk.norm_residual_backward(z, z, z, z, post=w, pre=w)
    assert not any(v.any() for v in g.values() if v is not None)


def test_no_tokens_another_stream_and_repeats(bk):
    import torch

    x, h, dy, dz, a = _make(0, 64, "float32", "rms", 1)
    y, z = bk.norm_residual(x, h, **a)
    g = bk.norm_residual_backward(dy, dz, y, h, **a)
    assert y.shape == z.shape == (0, 64) and not g["post"].any() and not g["gate"].any() and g["X"].shape == (0, 64)
    x, h, dy, dz, a = _make(900, 520, "bfloat16", "layer", 3)
    here, back = bk.norm_residual(x, h, **a, kind="layer"), bk.norm_residual_backward(dy, dz, x, h, **a, kind="layer")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = bk.norm_residual(x, h, **a, kind="layer", stream=side)
    back2 = bk.norm_residual_backward(dy, dz, x, h, **a, kind="layer", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(here, there))
    assert all(torch.equal(back[k], back2[k]) for k in back)


def test_refusals(bk):
    import torch

    x, h, dy, dz, a = _make(6, 64, "float32", "rms", 1)
    w = a["post"]
    for call in (lambda: bk.norm_residual(x, h[:5]), lambda: bk.norm_residual(x, h.half()), lambda: bk.norm_residual(x.cpu(), h),
                 lambda: bk.norm_residual(x, h, post=w[:5]), lambda: bk.norm_residual(x, h, post=w.half()),
                 lambda: bk.norm_residual(x, h, gate=torch.ones((4, 64), device="cuda")),
                 lambda: bk.norm_residual(x, h, gate=torch.ones((2, 64), device="cuda").half()),
                 lambda: bk.norm_residual(x, None, post=w), lambda: bk.norm_residual(x, h, kind="batch"),
                 lambda: bk.norm_residual(x, h, post=w, post_bias=w), lambda: bk.norm_residual(x, h, codes=True),
                 lambda: bk.norm_residual(x, h, pre_bias=w, kind="layer"), lambda: bk.norm_residual(x[0], h[0]),
                 lambda: bk.norm_residual(x.t(), h.t()),
                 lambda: bk.norm_residual_backward(None, None, x, h), lambda: bk.norm_residual_backward(dy, dz, x, h),
                 lambda: bk.norm_residual_backward(dy[:3], None, x, h)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):  # wider than 32768
        wide = torch.zeros((1, 32769), device="cuda")
        bk.norm_residual(wide, wide)
